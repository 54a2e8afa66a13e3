"""Batch-invariant LM-head token log-probabilities on GB300 (sm_103a).

A thin ctypes binding over ``liblmhead.so`` (C ABI declared in
``include/lmhead.h``). The functions keep the C names; they take torch
tensors, check dtypes/devices, allocate outputs and workspace with torch when
they are not given, and pass raw device pointers and the current CUDA stream
to the library. Every step of the computation runs in the library's CUDA
kernels: there is no Python, PyTorch or CPU path for any of them, and a
missing library raises instead of falling back.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

from ._build import LIB_PATH, build  # noqa: F401

LMH_OK = 0
LMH_ERR_INVALID_ARG = 1
LMH_ERR_ALIGNMENT = 2
LMH_ERR_WORKSPACE = 3
LMH_ERR_UNSUPPORTED_DEVICE = 4
LMH_ERR_LAUNCH = 5
LMH_ERR_DEVICE_TIMEOUT = 6
ERROR_NAMES = {
    0: "LMH_OK",
    1: "LMH_ERR_INVALID_ARG",
    2: "LMH_ERR_ALIGNMENT",
    3: "LMH_ERR_WORKSPACE",
    4: "LMH_ERR_UNSUPPORTED_DEVICE",
    5: "LMH_ERR_LAUNCH",
    6: "LMH_ERR_DEVICE_TIMEOUT",
}

LMH_OP_FWD = 0
LMH_OP_BWD = 1
LMH_OP_LOGITS = 2

# Exported C symbols and their signatures (argtypes, restype).
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_F = ctypes.c_float
SIGNATURES = {
    "lmhead_workspace_size": ([ctypes.c_int, _I64, _I64, _I64], ctypes.c_size_t),
    "lmhead_logprob_fwd": ([_P, _P, _P, _I64, _I64, _I64, _F, _P, _P, _P, _P, ctypes.c_size_t, _P],
                           ctypes.c_int),
    "lmhead_logprob_bwd": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _F, _P, _P, _P, ctypes.c_size_t,
                            _P], ctypes.c_int),
    "logprob_from_logits": ([_P, _P, _I64, _I64, _F, _P, _P, _P, _P], ctypes.c_int),
    "lmhead_logprob_fwd_stats": ([_P, _P, _P, _I64, _I64, _I64, _F, _P, _P, _P, _P, _P,
                                  ctypes.c_size_t, _P], ctypes.c_int),
    "logprob_from_logits_stats": ([_P, _P, _I64, _I64, _F, _P, _P, _P, _P, _P], ctypes.c_int),
    "logprob_from_logits_div": ([_P, _P, _I64, _I64, _F, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "lmhead_logprob_fwd_partials": ([_P, _P, _P, _I64, _I64, _I64, _I64, _F, _P, _P, _P, _P, _P],
                                    ctypes.c_int),
    "lmhead_logprob_merge": ([_P, _P, _P, _P, _P, _I64, _I64, _P, _P, _P, _P], ctypes.c_int),
    "lmhead_logprob_fwd_host": ([_P, _P, _P, _I64, _I64, _I64, _F, _P, _P, _P, _P, _P, _P, _P, _P,
                                 _P, ctypes.c_size_t, _P, _P], ctypes.c_int),
    "lmhead_last_error_string": ([], ctypes.c_char_p),
    "lmhead_abi_version": ([], ctypes.c_int),
    "lmhead_kernel_launches": ([], ctypes.c_ulonglong),
    "lmhead_timing_enable": ([ctypes.c_int], ctypes.c_int),
    "lmhead_timing_read": ([ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_float), ctypes.c_int,
                            ctypes.POINTER(ctypes.c_int)], ctypes.c_int),
    "lmhead_timing_kind_name": ([ctypes.c_int], ctypes.c_char_p),
    "lmhead_device_status": ([_P, ctypes.POINTER(ctypes.c_uint)], ctypes.c_int),
    "lmhead_selftest_wait_timeout": ([ctypes.c_uint64, _P], ctypes.c_int),
    "lmhead_selftest_division": ([_F, ctypes.POINTER(ctypes.c_int), _P], ctypes.c_int),
    "lmhead_engine_gemm": ([_P, _P, _I64, _I64, _I64, ctypes.c_int, _P, _P], ctypes.c_int),
    "lmhead_logprob_entropy_bwd": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F, _P, _P, _P,
                                    ctypes.c_size_t, _P], ctypes.c_int),
    "lmhead_logprob_fwd_noalloc": ([_P, _P, _P, _I64, _I64, _I64, _F, _P, _P, _P, _P],
                                   ctypes.c_int),
    "lmhead_logprob_bwd_chunked": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F, _I64, _P, _P,
                                    _P, ctypes.c_size_t, _P], ctypes.c_int),
    "lmhead_workspace_size_bwd": ([_I64, _I64, _I64, _I64], ctypes.c_size_t),
    "lmhead_logprob_bwd_shard": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _F, _P, _P,
                                  _P, ctypes.c_size_t, _P], ctypes.c_int),
    "lmhead_sum_ranks_bf16": ([_P, _I64, _I64, _P, _P], ctypes.c_int),
    "lmhead_quantize_fp8": ([_P, _I64, _I64, _I64, ctypes.c_int, _P, _P, _P], ctypes.c_int),
    "lmhead_logits_fp8": ([_P, _P, _P, _P, _I64, _I64, _I64, _P, _I64, _P], ctypes.c_int),
    "lmhead_sample": ([_P, _I64, _I64, _I64, _F, _P, ctypes.c_int32, _P, _F, _P, _F, _P, _P, _P, _P,
                       _P], ctypes.c_int),
    "lmhead_rmsnorm_fp8": ([_P, _P, _P, _I64, _I64, _I64, _I64, _F, _P, _I64, _P, _P, _P],
                           ctypes.c_int),
    "lmhead_quantize_mxfp4": ([_P, _I64, _I64, _I64, _P, _P, _P], ctypes.c_int),
    "lmhead_dequantize_mxfp4": ([_P, _P, _I64, _I64, _P, _I64, _P], ctypes.c_int),
    "lmhead_logits_mxfp4": ([_P, _P, _P, _P, _I64, _I64, _I64, _P, _I64, _P], ctypes.c_int),
    "lmhead_top_logprobs": ([_P, _I64, _I64, _I64, _F, _P, _P, _I64, _I64, _P, _P, _P, _P, _P],
                            ctypes.c_int),
}

_lib_handle: Optional[ctypes.CDLL] = None


class LMHeadError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn}: {ERROR_NAMES.get(code, code)}: {msg}")
        self.code = code


def library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load liblmhead.so (built by ``build()``); raises if it is missing."""
    global _lib_handle
    if _lib_handle is not None and path is None:
        return _lib_handle
    p = path or os.environ.get("LMHEAD_LIB") or str(LIB_PATH)
    if not os.path.exists(p):
        raise RuntimeError(f"liblmhead.so not found at {p}; run invariant_lm_head_gb300.build()")
    lib = ctypes.CDLL(p)
    for name, (args, res) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    if path is None:
        _lib_handle = lib
    return lib


def _check(fn: str, rc: int) -> None:
    if rc != LMH_OK:
        msg = library().lmhead_last_error_string().decode(errors="replace")
        raise LMHeadError(fn, rc, msg)


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


def _stream_ptr(stream) -> Optional[int]:
    if stream is not None:
        return stream.cuda_stream
    return _torch().cuda.current_stream().cuda_stream


def _launch_on(t, name: str, stream):
    """(handle, empty) of the stream that a call on t's device runs on (None: the current one).

    A kernel runs on the current device. Addresses of the host or of another device
    must never reach it, nor work be put on another device's stream. Every other
    tensor of a call is on t's device. empty is torch.empty for what the call writes.
    """
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name} must be on a CUDA device, got {t.device}")
    torch = _torch()
    current = torch.cuda.current_device()
    if device != current:
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{current}")
    if stream is None:
        # the handle without a Stream object around it (0.2 us instead of 2.8, of a
        # short call's ten)
        return torch._C._cuda_getCurrentRawStream(current), torch.empty
    if stream.device.index != current:
        raise ValueError(f"stream is on {stream.device}, but the current device is cuda:{current}")

    def empty(*size, **options):
        # The memory is the call's stream's: the current stream's may still be in use by
        # work ahead of the call, and a workspace would go back to it, free to be written,
        # while the call runs. What the current stream does with an output before it is
        # dropped is waited for as well.
        with torch.cuda.stream(stream):
            t = torch.empty(*size, **options)
        t.record_stream(torch.cuda.current_stream())
        return t

    return stream.cuda_stream, empty


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(t, name: str, dtype, device, ndim: int):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-D tensor")


def lmhead_workspace_size(op: int, T: int, H: int, V: int) -> int:
    n = library().lmhead_workspace_size(op, T, H, V)
    if n == ctypes.c_size_t(-1).value:
        _check("lmhead_workspace_size", LMH_ERR_INVALID_ARG)
    return n


def _workspace(op, T, H, V, workspace, device, empty):
    need = lmhead_workspace_size(op, T, H, V)
    if workspace is None:
        workspace = empty(max(need, 16), dtype=_torch().uint8, device=device)
    return workspace, workspace.numel() * workspace.element_size()


def lmhead_logprob_fwd(hidden, weight, labels, inv_temperature: float = 1.0, *, out_logprob=None,
                       out_entropy=None, out_lse=None, want_entropy: bool = True,
                       want_lse: bool = False, workspace=None, stream=None):
    """Fused LM-head forward. Returns (logprob, entropy or None, lse or None), f32 [T]."""
    return _fwd("lmhead_logprob_fwd", hidden, weight, labels, inv_temperature, out_logprob,
                out_entropy, out_lse, None, want_entropy, want_lse, False, workspace, stream)[:3]


def lmhead_logprob_fwd_stats(hidden, weight, labels, inv_temperature: float = 1.0, *,
                             out_logprob=None, out_entropy=None, out_lse=None, out_sum_p2=None,
                             want_entropy: bool = True, want_lse: bool = False, workspace=None,
                             stream=None):
    """Fused forward with sum_pi_squared. Returns (logprob, entropy, lse, sum_p2)."""
    return _fwd("lmhead_logprob_fwd_stats", hidden, weight, labels, inv_temperature, out_logprob,
                out_entropy, out_lse, out_sum_p2, want_entropy, want_lse, True, workspace, stream)


def lmhead_logprob_fwd_host(hidden_host, weight_host, labels_host, inv_temperature: float = 1.0,
                            *, hidden, weight, labels, out_logprob=None, out_entropy=None,
                            out_lse=None, out_logprob_host=None, out_entropy_host=None,
                            want_entropy: bool = True, want_lse: bool = True, workspace=None,
                            stream=None, copy_stream=None):
    """Fused forward from host inputs, copies overlapped with the forward.

    hidden_host, weight_host, labels_host are CPU tensors (page-locked for the
    copies to overlap); hidden, weight, labels are device tensors of the same
    shapes that the call fills. out_logprob_host / out_entropy_host (CPU f32
    [T] or None) receive the results in stream order. copy_stream is a
    torch.cuda.Stream or None (the library's own). Returns (logprob, entropy
    or None, lse or None) on the device.
    """
    torch = _torch()
    dev = hidden.device
    _need(hidden, "hidden", torch.bfloat16, dev, 2)
    _need(weight, "weight", torch.bfloat16, dev, 2)
    _need(labels, "labels", torch.int32, dev, 1)
    cpu = torch.device("cpu")
    _need(hidden_host, "hidden_host", torch.bfloat16, cpu, 2)
    _need(weight_host, "weight_host", torch.bfloat16, cpu, 2)
    _need(labels_host, "labels_host", torch.int32, cpu, 1)
    T, H = hidden.shape
    V = weight.shape[0]
    if (tuple(hidden_host.shape) != (T, H) or tuple(weight_host.shape) != (V, H)
            or weight.shape[1] != H or labels.shape[0] != T or labels_host.shape[0] != T):
        raise ValueError("shape mismatch between the host and device inputs")
    for t, n in ((out_logprob_host, "out_logprob_host"), (out_entropy_host, "out_entropy_host")):
        if t is not None:
            _need(t, n, torch.float32, cpu, 1)
    st, empty = _launch_on(hidden, "hidden", stream)
    if out_logprob is None:
        out_logprob = empty(T, dtype=torch.float32, device=dev)
    if out_entropy is None and (want_entropy or out_entropy_host is not None):
        out_entropy = empty(T, dtype=torch.float32, device=dev)
    if out_lse is None and want_lse:
        out_lse = empty(T, dtype=torch.float32, device=dev)
    ws, ws_bytes = _workspace(LMH_OP_FWD, T, H, V, workspace, dev, empty)
    cs = None if copy_stream is None else ctypes.c_void_p(copy_stream.cuda_stream)
    rc = library().lmhead_logprob_fwd_host(
        _ptr(hidden_host), _ptr(weight_host), _ptr(labels_host), T, H, V, float(inv_temperature),
        _ptr(hidden), _ptr(weight), _ptr(labels), _ptr(out_logprob), _ptr(out_entropy),
        _ptr(out_lse), _ptr(out_logprob_host), _ptr(out_entropy_host), _ptr(ws), ws_bytes, st,
        cs)
    _check("lmhead_logprob_fwd_host", rc)
    return out_logprob, out_entropy, out_lse


def _fwd(name, hidden, weight, labels, inv_temperature, out_logprob, out_entropy, out_lse,
         out_sum_p2, want_entropy, want_lse, want_sum_p2, workspace, stream):
    torch = _torch()
    dev = hidden.device
    _need(hidden, "hidden", torch.bfloat16, dev, 2)
    _need(weight, "weight", torch.bfloat16, dev, 2)
    _need(labels, "labels", torch.int32, dev, 1)
    T, H = hidden.shape
    V = weight.shape[0]
    if weight.shape[1] != H or labels.shape[0] != T:
        raise ValueError("shape mismatch between hidden, weight and labels")
    st, empty = _launch_on(hidden, "hidden", stream)
    if out_logprob is None:
        out_logprob = empty(T, dtype=torch.float32, device=dev)
    if out_entropy is None and want_entropy:
        out_entropy = empty(T, dtype=torch.float32, device=dev)
    if out_lse is None and want_lse:
        out_lse = empty(T, dtype=torch.float32, device=dev)
    if out_sum_p2 is None and want_sum_p2:
        out_sum_p2 = empty(T, dtype=torch.float32, device=dev)
    ws, ws_bytes = _workspace(LMH_OP_FWD, T, H, V, workspace, dev, empty)
    lib = library()
    args = [_ptr(hidden), _ptr(weight), _ptr(labels), T, H, V, float(inv_temperature),
            _ptr(out_logprob), _ptr(out_entropy), _ptr(out_lse)]
    if name == "lmhead_logprob_fwd_stats":
        args.append(_ptr(out_sum_p2))
    rc = getattr(lib, name)(*args, _ptr(ws), ws_bytes, st)
    _check(name, rc)
    return out_logprob, out_entropy, out_lse, out_sum_p2


def lmhead_logprob_bwd(hidden, weight, labels, grad_logprob, inv_temperature: float = 1.0, *,
                       lse=None, grad_hidden=None, grad_weight=None, workspace=None, stream=None):
    """Fused backward. Returns (grad_hidden bf16 [T, H], grad_weight f32 [V, H])."""
    torch = _torch()
    dev = hidden.device
    _need(hidden, "hidden", torch.bfloat16, dev, 2)
    _need(weight, "weight", torch.bfloat16, dev, 2)
    _need(labels, "labels", torch.int32, dev, 1)
    _need(grad_logprob, "grad_logprob", torch.float32, dev, 1)
    if lse is not None:
        _need(lse, "lse", torch.float32, dev, 1)
    st, empty = _launch_on(hidden, "hidden", stream)
    T, H = hidden.shape
    V = weight.shape[0]
    if grad_hidden is None:
        grad_hidden = empty(T, H, dtype=torch.bfloat16, device=dev)
    if grad_weight is None:
        grad_weight = empty(V, H, dtype=torch.float32, device=dev)
    ws, ws_bytes = _workspace(LMH_OP_BWD, T, H, V, workspace, dev, empty)
    rc = library().lmhead_logprob_bwd(_ptr(hidden), _ptr(weight), _ptr(labels), _ptr(grad_logprob),
                                      _ptr(lse), T, H, V, float(inv_temperature), _ptr(grad_hidden),
                                      _ptr(grad_weight), _ptr(ws), ws_bytes, st)
    _check("lmhead_logprob_bwd", rc)
    return grad_hidden, grad_weight


def lmhead_logprob_entropy_bwd(hidden, weight, labels, grad_logprob, grad_entropy,
                               inv_temperature: float = 1.0, *, lse=None, entropy=None,
                               grad_hidden=None, grad_weight=None, workspace=None, stream=None):
    """Backward of sum g*logprob + gH*entropy. Returns (grad_hidden bf16, grad_weight f32)."""
    torch = _torch()
    dev = hidden.device
    _need(hidden, "hidden", torch.bfloat16, dev, 2)
    _need(weight, "weight", torch.bfloat16, dev, 2)
    _need(labels, "labels", torch.int32, dev, 1)
    for t, n in ((grad_logprob, "grad_logprob"), (grad_entropy, "grad_entropy"), (lse, "lse"),
                 (entropy, "entropy")):
        if t is not None:
            _need(t, n, torch.float32, dev, 1)
    st, empty = _launch_on(hidden, "hidden", stream)
    T, H = hidden.shape
    V = weight.shape[0]
    if grad_hidden is None:
        grad_hidden = empty(T, H, dtype=torch.bfloat16, device=dev)
    if grad_weight is None:
        grad_weight = empty(V, H, dtype=torch.float32, device=dev)
    ws, ws_bytes = _workspace(LMH_OP_BWD, T, H, V, workspace, dev, empty)
    rc = library().lmhead_logprob_entropy_bwd(
        _ptr(hidden), _ptr(weight), _ptr(labels), _ptr(grad_logprob), _ptr(grad_entropy),
        _ptr(lse), _ptr(entropy), T, H, V, float(inv_temperature), _ptr(grad_hidden),
        _ptr(grad_weight), _ptr(ws), ws_bytes, st)
    _check("lmhead_logprob_entropy_bwd", rc)
    return grad_hidden, grad_weight


def lmhead_workspace_size_bwd(T: int, H: int, V: int, row_chunk: int) -> int:
    """Workspace bytes of lmhead_logprob_bwd_chunked."""
    n = library().lmhead_workspace_size_bwd(T, H, V, row_chunk)
    if n == ctypes.c_size_t(-1).value:
        _check("lmhead_workspace_size_bwd", LMH_ERR_INVALID_ARG)
    return n


def lmhead_logprob_bwd_chunked(hidden, weight, labels, grad_logprob, inv_temperature: float = 1.0,
                               *, row_chunk: int, grad_entropy=None, lse=None, entropy=None,
                               grad_hidden=None, grad_weight=None, workspace=None, stream=None):
    """Backward with a chosen row chunk (bounded workspace). Returns (grad_hidden, grad_weight)."""
    torch = _torch()
    dev = hidden.device
    _need(hidden, "hidden", torch.bfloat16, dev, 2)
    _need(weight, "weight", torch.bfloat16, dev, 2)
    _need(labels, "labels", torch.int32, dev, 1)
    for t, n in ((grad_logprob, "grad_logprob"), (grad_entropy, "grad_entropy"), (lse, "lse"),
                 (entropy, "entropy")):
        if t is not None:
            _need(t, n, torch.float32, dev, 1)
    st, empty = _launch_on(hidden, "hidden", stream)
    T, H = hidden.shape
    V = weight.shape[0]
    if grad_hidden is None:
        grad_hidden = empty(T, H, dtype=torch.bfloat16, device=dev)
    if grad_weight is None:
        grad_weight = empty(V, H, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = empty(max(lmhead_workspace_size_bwd(T, H, V, row_chunk), 16),
                          dtype=torch.uint8, device=dev)
    rc = library().lmhead_logprob_bwd_chunked(
        _ptr(hidden), _ptr(weight), _ptr(labels), _ptr(grad_logprob), _ptr(grad_entropy),
        _ptr(lse), _ptr(entropy), T, H, V, float(inv_temperature), int(row_chunk),
        _ptr(grad_hidden), _ptr(grad_weight), _ptr(workspace),
        workspace.numel() * workspace.element_size(), st)
    _check("lmhead_logprob_bwd_chunked", rc)
    return grad_hidden, grad_weight


def lmhead_logprob_bwd_shard(hidden, weight_shard, labels, grad_logprob, lse, v_offset: int,
                             inv_temperature: float = 1.0, *, grad_entropy=None, entropy=None,
                             grad_hidden_part=None, grad_weight=None, workspace=None, stream=None):
    """One vocab shard's backward (see include/lmhead.h).

    lse (and entropy, with grad_entropy) are the whole vocabulary's, f32 [T].
    Returns (grad_hidden_part f32 [T, H], grad_weight f32 [V_shard, H]).
    """
    torch = _torch()
    dev = hidden.device
    _need(hidden, "hidden", torch.bfloat16, dev, 2)
    _need(weight_shard, "weight_shard", torch.bfloat16, dev, 2)
    _need(labels, "labels", torch.int32, dev, 1)
    for t, n in ((grad_logprob, "grad_logprob"), (grad_entropy, "grad_entropy"), (lse, "lse"),
                 (entropy, "entropy")):
        if t is not None:
            _need(t, n, torch.float32, dev, 1)
    st, empty = _launch_on(hidden, "hidden", stream)
    T, H = hidden.shape
    V = weight_shard.shape[0]
    if grad_hidden_part is None:
        grad_hidden_part = empty(T, H, dtype=torch.float32, device=dev)
    if grad_weight is None:
        grad_weight = empty(V, H, dtype=torch.float32, device=dev)
    ws, ws_bytes = _workspace(LMH_OP_BWD, T, H, V, workspace, dev, empty)
    rc = library().lmhead_logprob_bwd_shard(
        _ptr(hidden), _ptr(weight_shard), _ptr(labels), _ptr(grad_logprob), _ptr(grad_entropy),
        _ptr(lse), _ptr(entropy), T, H, V, int(v_offset), float(inv_temperature),
        _ptr(grad_hidden_part), _ptr(grad_weight), _ptr(ws), ws_bytes, st)
    _check("lmhead_logprob_bwd_shard", rc)
    return grad_hidden_part, grad_weight


def lmhead_sum_ranks_bf16(parts, *, out=None, stream=None):
    """bf16 of the rank-ordered sum of parts [n, ...] (f32) over its first axis."""
    torch = _torch()
    dev = parts.device
    if not isinstance(parts, torch.Tensor) or parts.dtype != torch.float32:
        raise TypeError("parts must be a float32 tensor")
    if parts.device != dev or not parts.is_contiguous() or parts.dim() < 2:
        raise ValueError("parts must be a contiguous tensor [n, ...]")
    st, empty = _launch_on(parts, "parts", stream)
    n = parts.shape[0]
    count = parts[0].numel()
    if out is None:
        out = empty(parts.shape[1:], dtype=torch.bfloat16, device=dev)
    if out.dtype != torch.bfloat16 or out.numel() != count or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 tensor of parts[0]'s size")
    rc = library().lmhead_sum_ranks_bf16(_ptr(parts), n, count, _ptr(out), st)
    _check("lmhead_sum_ranks_bf16", rc)
    return out


def logprob_from_logits(logits, labels, inv_temperature: float = 1.0, *, out_logprob=None,
                        out_entropy=None, out_lse=None, want_entropy: bool = True,
                        want_lse: bool = False, stream=None):
    """Sampler formula on bf16 logits [T, V]. Returns (logprob, entropy or None, lse or None)."""
    return _logits("logprob_from_logits", logits, labels, inv_temperature, out_logprob,
                   out_entropy, out_lse, None, want_entropy, want_lse, False, stream)[:3]


def logprob_from_logits_stats(logits, labels, inv_temperature: float = 1.0, *, out_logprob=None,
                              out_entropy=None, out_lse=None, out_sum_p2=None,
                              want_entropy: bool = True, want_lse: bool = False, stream=None):
    """Sampler formula with sum_pi_squared. Returns (logprob, entropy, lse, sum_p2)."""
    return _logits("logprob_from_logits_stats", logits, labels, inv_temperature, out_logprob,
                   out_entropy, out_lse, out_sum_p2, want_entropy, want_lse, True, stream)


def logprob_from_logits_div(logits, labels, temperature=1.0, *, out_logprob=None,
                            out_entropy=None, out_lse=None, out_sum_p2=None,
                            want_entropy: bool = True, want_lse: bool = False,
                            want_sum_p2: bool = False, stream=None):
    """Sampler formula with the temperature as an fp32 division, z = logits / t.

    temperature is a float (one t for every row) or an f32 tensor [T] of
    per-row temperatures on the logits' device. Returns (logprob, entropy,
    lse, sum_p2), the ones not asked for None.
    """
    torch = _torch()
    row_t = None
    t = 1.0
    if isinstance(temperature, torch.Tensor):
        _need(temperature, "temperature", torch.float32, logits.device, 1)
        if temperature.shape[0] != logits.shape[0]:
            raise ValueError("temperature must have one value per row")
        row_t = temperature
    else:
        t = float(temperature)
    return _logits("logprob_from_logits_div", logits, labels, t, out_logprob, out_entropy,
                   out_lse, out_sum_p2, want_entropy, want_lse, want_sum_p2, stream, row_t=row_t)


def _logits(name, logits, labels, inv_temperature, out_logprob, out_entropy, out_lse, out_sum_p2,
            want_entropy, want_lse, want_sum_p2, stream, row_t=None):
    torch = _torch()
    dev = logits.device
    _need(logits, "logits", torch.bfloat16, dev, 2)
    _need(labels, "labels", torch.int32, dev, 1)
    st, empty = _launch_on(logits, "logits", stream)
    T, V = logits.shape
    if out_logprob is None:
        out_logprob = empty(T, dtype=torch.float32, device=dev)
    if out_entropy is None and want_entropy:
        out_entropy = empty(T, dtype=torch.float32, device=dev)
    if out_lse is None and want_lse:
        out_lse = empty(T, dtype=torch.float32, device=dev)
    if out_sum_p2 is None and want_sum_p2:
        out_sum_p2 = empty(T, dtype=torch.float32, device=dev)
    args = [_ptr(logits), _ptr(labels), T, V, float(inv_temperature)]
    if name == "logprob_from_logits_div":
        args.append(_ptr(row_t))
    args += [_ptr(out_logprob), _ptr(out_entropy), _ptr(out_lse)]
    if name in ("logprob_from_logits_stats", "logprob_from_logits_div"):
        args.append(_ptr(out_sum_p2))
    rc = getattr(library(), name)(*args, st)
    _check(name, rc)
    return out_logprob, out_entropy, out_lse, out_sum_p2


def lmhead_logprob_fwd_partials(hidden, weight_shard, labels, v_offset: int,
                                inv_temperature: float = 1.0, *, part_m, part_s, part_u,
                                label_logit, stream=None):
    """One vocab shard's forward statistics (see include/lmhead.h).

    part_m, part_s, part_u: f32 [ceil(V_shard / 1024), T] views into the
    whole-vocabulary planes at chunk v_offset / 1024; label_logit f32 [T].
    """
    torch = _torch()
    dev = hidden.device
    _need(hidden, "hidden", torch.bfloat16, dev, 2)
    _need(weight_shard, "weight_shard", torch.bfloat16, dev, 2)
    _need(labels, "labels", torch.int32, dev, 1)
    T, H = hidden.shape
    V = weight_shard.shape[0]
    n = -(-V // 1024)
    for t, nm in ((part_m, "part_m"), (part_s, "part_s"), (part_u, "part_u")):
        _need(t, nm, torch.float32, dev, 2)
        if tuple(t.shape) != (n, T):
            raise ValueError(f"{nm} must be [{n}, {T}]")
    _need(label_logit, "label_logit", torch.float32, dev, 1)
    st, _ = _launch_on(hidden, "hidden", stream)
    rc = library().lmhead_logprob_fwd_partials(
        _ptr(hidden), _ptr(weight_shard), _ptr(labels), T, H, V, int(v_offset),
        float(inv_temperature), _ptr(part_m), _ptr(part_s), _ptr(part_u), _ptr(label_logit), st)
    _check("lmhead_logprob_fwd_partials", rc)


def lmhead_logprob_merge(part_m, part_s, part_u, label_logit, labels, V: int, *,
                         out_logprob=None, out_entropy=None, out_lse=None, stream=None):
    """Merge whole-vocabulary planes into (logprob, entropy, lse), f32 [T]."""
    torch = _torch()
    dev = labels.device
    st, empty = _launch_on(labels, "labels", stream)
    T = labels.shape[0]
    out_logprob = empty(T, device=dev) if out_logprob is None else out_logprob
    out_entropy = empty(T, device=dev) if out_entropy is None else out_entropy
    out_lse = empty(T, device=dev) if out_lse is None else out_lse
    n = -(-int(V) // 1024)
    for t, nm in ((part_m, "part_m"), (part_s, "part_s"), (part_u, "part_u")):
        _need(t, nm, torch.float32, dev, 2)
        if tuple(t.shape) != (n, T):
            raise ValueError(f"{nm} must be [{n}, {T}]")
    rc = library().lmhead_logprob_merge(
        _ptr(part_m), _ptr(part_s), _ptr(part_u), _ptr(label_logit), _ptr(labels), T, int(V),
        _ptr(out_logprob), _ptr(out_entropy), _ptr(out_lse), st)
    _check("lmhead_logprob_merge", rc)
    return out_logprob, out_entropy, out_lse


def _need_rows(t, name: str, dtype, device, shape=None) -> int:
    """A matrix whose rows are contiguous, at any row stride; returns the stride."""
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    rows, cols = t.shape
    if shape is not None and (rows, cols) != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    ld, inner = t.stride()
    if cols > 1 and inner != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if rows <= 1:  # one row has no stride to respect
        return -(-cols // 8) * 8
    if ld < cols:
        raise ValueError(f"{name} must have rows that do not overlap")
    return ld


def _need_out(t, name: str, dtype, device, shape):
    _need(t, name, dtype, device, len(shape))
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}")


def lmhead_quantize_fp8(x, block_rows: int = 1, *, out=None, out_scale=None, stream=None):
    """Block quantisation of a bf16 matrix to e4m3 (see include/lmhead.h).

    x bf16 [rows, cols] (rows may be strided), blocks of block_rows (1 or 128)
    x 128. Returns (q float8_e4m3fn [rows, cols], scale f32 [ceil(rows /
    block_rows), ceil(cols / 128)]).
    """
    torch = _torch()
    dev = x.device
    ld = _need_rows(x, "x", torch.bfloat16, dev)
    rows, cols = x.shape
    if block_rows != 1 and block_rows != 128:
        raise ValueError("block_rows must be 1 or 128")
    st, empty = _launch_on(x, "x", stream)
    shape = (-(-rows // block_rows), -(-cols // 128))
    if out is None:
        out = empty((rows, cols), dtype=torch.float8_e4m3fn, device=dev)
    else:
        _need_out(out, "out", torch.float8_e4m3fn, dev, (rows, cols))
    if out_scale is None:
        out_scale = empty(shape, dtype=torch.float32, device=dev)
    else:
        _need_out(out_scale, "out_scale", torch.float32, dev, shape)
    rc = library().lmhead_quantize_fp8(x.data_ptr(), rows, cols, ld, block_rows, out.data_ptr(),
                                       out_scale.data_ptr(), st)
    if rc:
        _check("lmhead_quantize_fp8", rc)
    return out, out_scale


def lmhead_logits_fp8(hidden_q, hidden_scale, weight_q, weight_scale, *, out_logits=None,
                      stream=None):
    """bf16 logits [T, V] of block-scaled e4m3 operands (see include/lmhead.h).

    hidden_q [T, H] with hidden_scale [T, ceil(H / 128)], weight_q [V, H] with
    weight_scale [ceil(V / 128), ceil(H / 128)], as lmhead_quantize_fp8 returns
    them with block_rows 1 and 128. out_logits may have strided rows.
    """
    torch = _torch()
    dev = hidden_q.device
    f8, f32 = torch.float8_e4m3fn, torch.float32
    _need(hidden_q, "hidden_q", f8, dev, 2)
    _need(weight_q, "weight_q", f8, dev, 2)
    T, H = hidden_q.shape
    V, weight_cols = weight_q.shape
    if weight_cols != H:
        raise ValueError("shape mismatch between hidden_q and weight_q")
    kb = -(-H // 128)
    _need_out(hidden_scale, "hidden_scale", f32, dev, (T, kb))
    _need_out(weight_scale, "weight_scale", f32, dev, (-(-V // 128), kb))
    st, empty = _launch_on(hidden_q, "hidden_q", stream)
    if out_logits is None:
        out_logits = empty((T, V), dtype=torch.bfloat16, device=dev)
        ld = V
    else:
        ld = _need_rows(out_logits, "out_logits", torch.bfloat16, dev, (T, V))
    rc = library().lmhead_logits_fp8(hidden_q.data_ptr(), hidden_scale.data_ptr(),
                                     weight_q.data_ptr(), weight_scale.data_ptr(), T, H, V,
                                     out_logits.data_ptr(), ld, st)
    if rc:
        _check("lmhead_logits_fp8", rc)
    return out_logits


def _setting(v, name: str, dtype, device, rows: int):
    """A sampler setting: (number, None), or (None, one value per row)."""
    if not isinstance(v, _torch().Tensor):
        return v, None
    _need(v, name, dtype, device, 1)
    if v.shape[0] != rows:
        raise ValueError(f"{name} must have one value per row")
    return 0, v.data_ptr()


def lmhead_sample(logits, uniform, temperature=1.0, *, top_k=0, top_p=1.0, min_p=0.0,
                  out_token=None, out_logprob=None, want_logprob: bool = True, stream=None):
    """One token per row of bf16 logits from a given uniform number (see include/lmhead.h).

    logits bf16 [T, V] (rows may be strided), uniform f32 [T] in [0, 1].
    temperature (0: greedy), top_k (0: off), top_p (1: off) and min_p (0: off)
    are numbers, or tensors [T] (f32; top_k int32) with one value per row.
    Returns (token int32 [T], logprob f32 [T] or None).
    """
    torch = _torch()
    dev = logits.device
    f32, i32 = torch.float32, torch.int32
    ld = _need_rows(logits, "logits", torch.bfloat16, dev)
    T, V = logits.shape
    _need(uniform, "uniform", f32, dev, 1)
    if uniform.shape[0] != T:
        raise ValueError("uniform must have one value per row")
    t, row_t = _setting(temperature, "temperature", f32, dev, T)
    k, row_k = _setting(top_k, "top_k", i32, dev, T)
    p, row_p = _setting(top_p, "top_p", f32, dev, T)
    m, row_m = _setting(min_p, "min_p", f32, dev, T)
    k = int(k)
    if not 0 <= k <= 0x7fffffff:
        raise ValueError("top_k must be in [0, 2^31)")
    st, empty = _launch_on(logits, "logits", stream)
    if out_token is None:
        out_token = empty((T,), dtype=i32, device=dev)
    else:
        _need_out(out_token, "out_token", i32, dev, (T,))
    if out_logprob is not None:
        _need_out(out_logprob, "out_logprob", f32, dev, (T,))
    elif want_logprob:
        out_logprob = empty((T,), dtype=f32, device=dev)
    rc = library().lmhead_sample(logits.data_ptr(), T, V, ld, t, row_t, k, row_k, p, row_p, m,
                                 row_m, uniform.data_ptr(), out_token.data_ptr(),
                                 _ptr(out_logprob), st)
    if rc:
        _check("lmhead_sample", rc)
    return out_token, out_logprob


# The five calls below check the usual arguments (plain tensors, on the current stream) in
# one expression, 2.6 us less of a short call's 16 than the checks that name what is
# wrong; anything else goes through those.

def lmhead_rmsnorm_fp8(x, weight, residual=None, *, eps: float = 1e-6, out=None, out_scale=None,
                       out_residual=None, want_residual: bool = True, stream=None):
    """RMS norm of x (+ residual), block-quantised to e4m3 (see include/lmhead.h).

    x and residual bf16 [rows, cols] (rows may be strided), weight bf16 [cols].
    Returns (q float8_e4m3fn [rows, cols], scale f32 [rows, ceil(cols / 128)], the
    bf16 sum x + residual or None), q and scale as lmhead_logits_fp8 takes them.
    out_residual may be residual or x itself; want_residual=False leaves the sum out.
    """
    torch = _torch()
    tensor, bf16, dev, size, index = torch.Tensor, torch.bfloat16, x.device, x.shape, x.get_device()
    if (stream is None and out is None and out_scale is None and out_residual is None
            and index >= 0 and x.dtype is bf16 and len(size) == 2 and x.is_contiguous()
            and isinstance(weight, tensor) and weight.dtype is bf16 and weight.shape == size[1:]
            and weight.is_contiguous() and weight.get_device() == index
            and (residual is None or isinstance(residual, tensor) and residual.dtype is bf16
                 and residual.shape == size and residual.is_contiguous()
                 and residual.get_device() == index)
            and torch.cuda.current_device() == index):
        rows, ld = size
        cols = ld_res = ld_out = ld
        st, empty = torch._C._cuda_getCurrentRawStream(index), torch.empty
    else:
        ld = _need_rows(x, "x", bf16, dev)
        rows, cols = size
        _need_out(weight, "weight", bf16, dev, (cols,))
        ld_res, ld_out = 0, cols
        if residual is not None:
            ld_res = _need_rows(residual, "residual", bf16, dev, (rows, cols))
        elif out_residual is not None:
            raise ValueError("out_residual needs a residual")
        if out is not None:
            _need_out(out, "out", torch.float8_e4m3fn, dev, (rows, cols))
        if out_scale is not None:
            _need_out(out_scale, "out_scale", torch.float32, dev, (rows, -(-cols // 128)))
        if out_residual is not None:
            ld_out = _need_rows(out_residual, "out_residual", bf16, dev, (rows, cols))
        st, empty = _launch_on(x, "x", stream)
    if out is None:
        out = empty(size, dtype=torch.float8_e4m3fn, device=dev)
    if out_scale is None:
        out_scale = empty((rows, -(-cols // 128)), dtype=torch.float32, device=dev)
    if out_residual is None and residual is not None and want_residual:
        out_residual = empty(size, dtype=bf16, device=dev)
    rc = library().lmhead_rmsnorm_fp8(
        x.data_ptr(), None if residual is None else residual.data_ptr(), weight.data_ptr(), rows,
        cols, ld, ld_res, eps, None if out_residual is None else out_residual.data_ptr(), ld_out,
        out.data_ptr(), out_scale.data_ptr(), st)
    if rc:
        _check("lmhead_rmsnorm_fp8", rc)
    return out, out_scale, out_residual


def _mxfp4_scale_shape(rows: int, cols: int):
    return (-(-rows // 128), -(-cols // 128), 32, 16)


def lmhead_quantize_mxfp4(x, *, out=None, out_scale=None, stream=None):
    """Microscaled 4-bit quantisation of a bf16 matrix (see include/lmhead.h).

    x bf16 [rows, cols] (rows may be strided), cols a multiple of 32. Returns (q
    uint8 [rows, cols / 2], two e2m1 elements a byte, scale uint8 [ceil(rows / 128),
    ceil(cols / 128), 32, 16]).
    """
    torch = _torch()
    u8, dev, size, index = torch.uint8, x.device, x.shape, x.get_device()
    if (stream is None and out is None and out_scale is None and index >= 0
            and x.dtype is torch.bfloat16 and len(size) == 2 and x.is_contiguous()
            and torch.cuda.current_device() == index):
        rows, cols = size
        ld = cols
        st, empty = torch._C._cuda_getCurrentRawStream(index), torch.empty
    else:
        ld = _need_rows(x, "x", torch.bfloat16, dev)
        rows, cols = size
        if out is not None:
            _need_out(out, "out", u8, dev, (rows, cols // 2))
        if out_scale is not None:
            _need_out(out_scale, "out_scale", u8, dev, _mxfp4_scale_shape(rows, cols))
        st, empty = _launch_on(x, "x", stream)
    if out is None:
        out = empty((rows, cols // 2), dtype=u8, device=dev)
    if out_scale is None:
        out_scale = empty(_mxfp4_scale_shape(rows, cols), dtype=u8, device=dev)
    rc = library().lmhead_quantize_mxfp4(x.data_ptr(), rows, cols, ld, out.data_ptr(),
                                         out_scale.data_ptr(), st)
    if rc:
        _check("lmhead_quantize_mxfp4", rc)
    return out, out_scale


def lmhead_dequantize_mxfp4(q, scale, *, out=None, stream=None):
    """The bf16 values [rows, cols] that lmhead_quantize_mxfp4's output stands for."""
    torch = _torch()
    u8, dev, size, index = torch.uint8, q.device, q.shape, q.get_device()
    if (stream is None and out is None and index >= 0 and q.dtype is u8 and len(size) == 2
            and q.is_contiguous() and isinstance(scale, torch.Tensor) and scale.dtype is u8
            and scale.get_device() == index
            and scale.shape == _mxfp4_scale_shape(size[0], 2 * size[1]) and scale.is_contiguous()
            and torch.cuda.current_device() == index):
        rows, cols = size[0], 2 * size[1]
        ld = cols
        st, empty = torch._C._cuda_getCurrentRawStream(index), torch.empty
    else:
        _need(q, "q", u8, dev, 2)
        rows, cols = size[0], 2 * size[1]
        _need_out(scale, "scale", u8, dev, _mxfp4_scale_shape(rows, cols))
        ld = cols
        if out is not None:
            ld = _need_rows(out, "out", torch.bfloat16, dev, (rows, cols))
        st, empty = _launch_on(q, "q", stream)
    if out is None:
        out = empty((rows, cols), dtype=torch.bfloat16, device=dev)
    rc = library().lmhead_dequantize_mxfp4(q.data_ptr(), scale.data_ptr(), rows, cols,
                                           out.data_ptr(), ld, st)
    if rc:
        _check("lmhead_dequantize_mxfp4", rc)
    return out


def lmhead_logits_mxfp4(hidden_q, hidden_scale, weight_q, weight_scale, *, out_logits=None,
                        stream=None):
    """bf16 logits [T, V] of two microscaled 4-bit operands (see include/lmhead.h).

    hidden_q [T, H / 2] with hidden_scale and weight_q [V, H / 2] with weight_scale,
    as lmhead_quantize_mxfp4 returns them. out_logits may have strided rows.
    """
    torch = _torch()
    tensor, u8, dev, index = torch.Tensor, torch.uint8, hidden_q.device, hidden_q.get_device()
    size = hidden_q.shape
    if (stream is None and out_logits is None and index >= 0 and hidden_q.dtype is u8
            and len(size) == 2 and hidden_q.is_contiguous() and isinstance(weight_q, tensor)
            and weight_q.dtype is u8 and weight_q.dim() == 2 and weight_q.shape[1] == size[1]
            and weight_q.is_contiguous() and weight_q.get_device() == index
            and isinstance(hidden_scale, tensor) and hidden_scale.dtype is u8
            and hidden_scale.shape == _mxfp4_scale_shape(size[0], 2 * size[1])
            and hidden_scale.is_contiguous() and hidden_scale.get_device() == index
            and isinstance(weight_scale, tensor) and weight_scale.dtype is u8
            and weight_scale.shape == _mxfp4_scale_shape(weight_q.shape[0], 2 * size[1])
            and weight_scale.is_contiguous() and weight_scale.get_device() == index
            and torch.cuda.current_device() == index):
        T, V, H = size[0], weight_q.shape[0], 2 * size[1]
        ld = V
        st, empty = torch._C._cuda_getCurrentRawStream(index), torch.empty
    else:
        _need(hidden_q, "hidden_q", u8, dev, 2)
        _need(weight_q, "weight_q", u8, dev, 2)
        T, V, H = size[0], weight_q.shape[0], 2 * size[1]
        if weight_q.shape[1] != size[1]:
            raise ValueError("shape mismatch between hidden_q and weight_q")
        _need_out(hidden_scale, "hidden_scale", u8, dev, _mxfp4_scale_shape(T, H))
        _need_out(weight_scale, "weight_scale", u8, dev, _mxfp4_scale_shape(V, H))
        ld = V
        if out_logits is not None:
            ld = _need_rows(out_logits, "out_logits", torch.bfloat16, dev, (T, V))
        st, empty = _launch_on(hidden_q, "hidden_q", stream)
    if out_logits is None:
        out_logits = empty((T, V), dtype=torch.bfloat16, device=dev)
    rc = library().lmhead_logits_mxfp4(hidden_q.data_ptr(), hidden_scale.data_ptr(),
                                       weight_q.data_ptr(), weight_scale.data_ptr(), T, H, V,
                                       out_logits.data_ptr(), ld, st)
    if rc:
        _check("lmhead_logits_mxfp4", rc)
    return out_logits


def lmhead_top_logprobs(logits, tokens=None, temperature=1.0, *, top: int = 20, out_logprob=None,
                        out_entropy=None, out_top_token=None, out_top_logprob=None,
                        want_entropy: bool = True, stream=None):
    """Log-probs of given tokens, the entropy, and the likeliest alternatives.

    logits bf16 [T, V] (rows may be strided), tokens int32 [T] or [T, n] (or None),
    temperature a number or f32 [T] (0 counts as 1), top the number of alternatives (0
    to 128). Returns (logprob f32, shaped as tokens, or None; entropy f32 [T] or None;
    top_token int32 [T, top]; top_logprob f32 [T, top]); see include/lmhead.h for masks.
    want_entropy=False saves the output, not the time.
    """
    torch = _torch()
    f32, i32, dev = torch.float32, torch.int32, logits.device
    size, index = logits.shape, logits.get_device()
    if not 0 <= top <= 128:
        raise ValueError("top must be in [0, 128]")
    per_row = isinstance(temperature, torch.Tensor)
    if (stream is None and out_logprob is None and out_entropy is None and out_top_token is None
            and out_top_logprob is None and index >= 0 and logits.dtype is torch.bfloat16
            and len(size) == 2 and logits.is_contiguous()
            and (tokens is None or isinstance(tokens, torch.Tensor) and tokens.dtype is i32
                 and 1 <= tokens.dim() <= 2 and tokens.shape[0] == size[0]
                 and tokens.is_contiguous() and tokens.get_device() == index)
            and (not per_row or temperature.dtype is f32 and temperature.shape == size[:1]
                 and temperature.is_contiguous() and temperature.get_device() == index)
            and torch.cuda.current_device() == index):
        T, V = size
        ld = V
        t, row_t = (0, temperature.data_ptr()) if per_row else (temperature, None)
        st, empty = torch._C._cuda_getCurrentRawStream(index), torch.empty
    else:
        ld = _need_rows(logits, "logits", torch.bfloat16, dev)
        T, V = size
        if tokens is not None:
            if not isinstance(tokens, torch.Tensor):
                raise TypeError("tokens must be a torch.Tensor")
            if tokens.dim() not in (1, 2):
                raise ValueError("tokens must be a 1-D or 2-D tensor")
            _need(tokens, "tokens", i32, dev, tokens.dim())
            if tokens.shape[0] != T:
                raise ValueError("tokens must have one row per row of logits")
            if out_logprob is not None:
                _need_out(out_logprob, "out_logprob", f32, dev, tuple(tokens.shape))
        elif out_logprob is not None:
            raise ValueError("out_logprob needs tokens")
        t, row_t = _setting(temperature, "temperature", f32, dev, T)
        if out_entropy is not None:
            _need_out(out_entropy, "out_entropy", f32, dev, (T,))
        if out_top_token is not None:
            _need_out(out_top_token, "out_top_token", i32, dev, (T, top))
        if out_top_logprob is not None:
            _need_out(out_top_logprob, "out_top_logprob", f32, dev, (T, top))
        st, empty = _launch_on(logits, "logits", stream)
    n_tokens = 0
    if tokens is not None:
        n_tokens = 1 if tokens.dim() == 1 else tokens.shape[1]
        if out_logprob is None:
            out_logprob = empty(tokens.shape, dtype=f32, device=dev)
    if out_entropy is None and want_entropy:
        out_entropy = empty((T,), dtype=f32, device=dev)
    if out_top_token is None:
        out_top_token = empty((T, top), dtype=i32, device=dev)
    if out_top_logprob is None:
        out_top_logprob = empty((T, top), dtype=f32, device=dev)
    rc = library().lmhead_top_logprobs(
        logits.data_ptr(), T, V, ld, t, row_t, None if tokens is None else tokens.data_ptr(),
        n_tokens, top, None if out_logprob is None else out_logprob.data_ptr(),
        None if out_entropy is None else out_entropy.data_ptr(), out_top_token.data_ptr(),
        out_top_logprob.data_ptr(), st)
    if rc:
        _check("lmhead_top_logprobs", rc)
    return out_logprob, out_entropy, out_top_token, out_top_logprob


_LOGPROB_FN = None
# Row chunk of the autograd backward (lmhead_logprob_bwd_chunked): at H = 3584,
# V = 152064 its workspace is 1.4 GB instead of 5.6 GB for 16384 rows.
AUTOGRAD_ROW_CHUNK = 4096


def _logprob_function():
    """The autograd Function behind lmhead_logprob, built on first use (torch
    is imported lazily so that the module loads without it)."""
    global _LOGPROB_FN
    if _LOGPROB_FN is not None:
        return _LOGPROB_FN
    torch = _torch()

    class _LMHeadLogprob(torch.autograd.Function):
        @staticmethod
        def forward(ctx, hidden, weight, labels, inv_temperature):
            lp, ent, lse = lmhead_logprob_fwd(hidden, weight, labels, inv_temperature,
                                              want_lse=True)
            ctx.save_for_backward(hidden, weight, labels, lse, ent)
            ctx.inv_temperature = inv_temperature
            ctx.set_materialize_grads(False)
            return lp, ent

        @staticmethod
        def backward(ctx, grad_logprob, grad_entropy):
            hidden, weight, labels, lse, ent = ctx.saved_tensors
            if grad_logprob is None and grad_entropy is None:
                return None, None, None, None
            s = ctx.inv_temperature
            g = None if grad_logprob is None else grad_logprob.float().contiguous()
            ge = None if grad_entropy is None else grad_entropy.float().contiguous()
            # rows in chunks of AUTOGRAD_ROW_CHUNK: a quarter of the default
            # backward's workspace, at no measurable cost in time
            gh, gw = lmhead_logprob_bwd_chunked(hidden, weight, labels, g, s,
                                                row_chunk=AUTOGRAD_ROW_CHUNK, grad_entropy=ge,
                                                lse=lse, entropy=ent if ge is not None else None)
            gw_out = None
            if ctx.needs_input_grad[1]:
                # the fp32 sum rounded once to the weight's bf16 by the library
                gw_out = lmhead_sum_ranks_bf16(gw.view(1, *gw.shape))
            del gw
            return (gh if ctx.needs_input_grad[0] else None, gw_out, None, None)

    _LOGPROB_FN = _LMHeadLogprob
    return _LOGPROB_FN


def lmhead_logprob(hidden, weight, labels, inv_temperature: float = 1.0):
    """Differentiable fused LM-head log-probs: (logprob, entropy), f32 [T].

    Forward is lmhead_logprob_fwd; backward is lmhead_logprob_bwd, or
    lmhead_logprob_entropy_bwd when the entropy output also receives a
    gradient. hidden bf16 [T, H] and weight bf16 [V, H] get bf16 gradients
    (grad_weight is accumulated in fp32 by the library and rounded once to
    bf16 by it; call lmhead_logprob_bwd directly to keep it in fp32). The
    backward runs in row chunks of AUTOGRAD_ROW_CHUNK. labels int32 [T] get
    none.
    """
    return _logprob_function().apply(hidden, weight, labels, float(inv_temperature))


def lmhead_kernel_launches() -> int:
    """Kernels launched by the library in this process so far."""
    return int(library().lmhead_kernel_launches())


def lmhead_timing_enable(on: bool = True) -> None:
    """Start (and clear) or stop per-launch event timing inside the library."""
    _check("lmhead_timing_enable", library().lmhead_timing_enable(1 if on else 0))


def lmhead_timing_read(capacity: int = 1 << 16):
    """[(kernel kind name, milliseconds)] for the launches recorded since enabling."""
    kinds = (ctypes.c_int * capacity)()
    ms = (ctypes.c_float * capacity)()
    n = ctypes.c_int(0)
    lib = library()
    _check("lmhead_timing_read", lib.lmhead_timing_read(kinds, ms, capacity, ctypes.byref(n)))
    return [(lib.lmhead_timing_kind_name(kinds[i]).decode(), float(ms[i])) for i in range(n.value)]


def lmhead_device_status(stream=None) -> int:
    """Synchronise the stream; return the device status word (raises on a timeout bit)."""
    bits = ctypes.c_uint(0)
    rc = library().lmhead_device_status(_stream_ptr(stream), ctypes.byref(bits))
    _check("lmhead_device_status", rc)
    return bits.value


def lmhead_selftest_wait_timeout(limit_ns: int = 1_000_000, stream=None) -> int:
    """Run the bounded-wait self-test; returns the library's status code (6 expected)."""
    return library().lmhead_selftest_wait_timeout(int(limit_ns), _stream_ptr(stream))


def lmhead_selftest_division(temperature: float, stream=None) -> int:
    """Number of bf16 inputs whose quotient in the division form differs from
    IEEE fp32 division by ``temperature`` (0 = bit-exact)."""
    n = ctypes.c_int(-1)
    _check("lmhead_selftest_division",
           library().lmhead_selftest_division(float(temperature), ctypes.byref(n),
                                              _stream_ptr(stream)))
    return int(n.value)


def lmhead_engine_gemm(A, B, out=None, a_kmajor: bool = True, b_kmajor: bool = True,
                       stream=None):
    """D = sum_k A[m,k] B[n,k] through the tensor-core engine; D f32 [M, N].

    A is [M, K] when a_kmajor else [K, M]; B is [N, K] when b_kmajor else [K, N].
    """
    torch = _torch()
    dev = A.device
    _need(A, "A", torch.bfloat16, dev, 2)
    _need(B, "B", torch.bfloat16, dev, 2)
    M, K = A.shape if a_kmajor else (A.shape[1], A.shape[0])
    N = B.shape[0] if b_kmajor else B.shape[1]
    layout = (0 if a_kmajor else 1) | (0 if b_kmajor else 2)
    st, empty = _launch_on(A, "A", stream)
    if out is None:
        out = empty(M, N, dtype=torch.float32, device=dev)
    rc = library().lmhead_engine_gemm(_ptr(A), _ptr(B), M, N, K, layout, _ptr(out), st)
    _check("lmhead_engine_gemm", rc)
    return out
