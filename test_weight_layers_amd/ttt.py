"""Thin Python binding of libttt.so (C ABI in include/ttt.h).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  Tensors must live on the current GPU; calls are asynchronous on
``torch.cuda.current_stream()``.  Errors raise ``TTTError`` with the library's
message.  There is no CPU fallback: if the library is missing, the first call
raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Sequence, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libttt.so")

TTT_F32, TTT_BF16 = 0, 1
OPT_FORCE_GENERAL, OPT_SPLITS, OPT_NS_UNFUSED = 0, 1, 2
KERNEL_KINDS = ("conv", "cast", "grad", "reduce", "ns", "apply", "gate", "delta", "residual", "orthogonalise",
                "attention", "norm", "adamw")
NORM_PRESERVE = 1
DELTA_ZERO_UNUSED = 1
ATTENTION_ZERO_UNUSED = 1
EXPORTS = ("ttt_last_error", "ttt_update_workspace_bytes", "ttt_apply_workspace_bytes", "ttt_update",
           "ttt_update_ex", "ttt_update_host_workspace_bytes", "ttt_update_host", "ttt_apply", "ttt_output_gate", "ttt_shortconv2d", "ttt_stream_workspace_bytes",
           "ttt_stream", "ttt_stream_ex", "ttt_set_option", "ttt_profile_enable", "ttt_profile_reset",
           "ttt_profile_read", "ttt_update_noalloc", "ttt_noalloc_scratch_bytes", "ttt_mfma_rate_probe",
           "ttt_delta_workspace_bytes", "ttt_delta", "ttt_delta_backward", "ttt_delta_step", "ttt_gated_residual",
           "ttt_gated_residual_backward_workspace_bytes", "ttt_gated_residual_backward",
           "ttt_orthogonalise_workspace_bytes", "ttt_orthogonalise", "ttt_window_attention_workspace_bytes",
           "ttt_window_attention", "ttt_window_attention_backward", "ttt_window_attention_step_workspace_bytes",
           "ttt_window_attention_step", "ttt_layer_norm", "ttt_layer_norm_backward_workspace_bytes",
           "ttt_layer_norm_backward", "ttt_adamw_check", "ttt_adamw_step")

_lib = None


class TTTError(RuntimeError):
    pass


class _AdamwTensor(ctypes.Structure):
    """ttt_adamw_tensor."""
    _fields_ = [(x, ctypes.c_void_p) for x in ("param", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scale",
                                               "exp_avg_sq_scale", "master")] + [("n", ctypes.c_int64)]


def load() -> ctypes.CDLL:
    """Load libttt.so once and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise TTTError(f"{LIB_PATH} is not built (run __graft_entry__.build())")
    L = ctypes.CDLL(LIB_PATH)
    i32, i64, f32, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    vp, szp, u32 = ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t), ctypes.c_uint32
    sig = {
        "ttt_last_error": (ctypes.c_char_p, []),
        "ttt_update_workspace_bytes": (ctypes.c_int, [i32, i32, i32, i64, i32, szp]),
        "ttt_apply_workspace_bytes": (ctypes.c_int, [i32, i32, i32, i64, i32, szp]),
        "ttt_stream_workspace_bytes": (ctypes.c_int, [i32, i32, i32, i64, i32, szp]),
        "ttt_update": (ctypes.c_int, [i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, i64, vp, i64, i64, f32, i32,
                                      i32, vp, vp, vp, sz, vp]),
        "ttt_update_ex": (ctypes.c_int, [i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, i64, vp, i64, i64, f32,
                                         i32, i32, u32, vp, vp, vp, sz, vp]),
        "ttt_update_noalloc": (ctypes.c_int, [i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, i64, vp, i64, i64, f32,
                                              i32, i32, u32, vp, vp, vp]),
        "ttt_noalloc_scratch_bytes": (ctypes.c_int, [szp]),
        "ttt_update_host_workspace_bytes": (ctypes.c_int, [i32, i32, i32, i64, i64, i32, szp]),
        "ttt_update_host": (ctypes.c_int, [i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, i64, vp, i64, i64, i64,
                                           f32, i32, i32, u32, vp, vp, vp, sz, vp]),
        "ttt_output_gate": (ctypes.c_int, [i32, vp, i64, vp, vp, f32, vp, i64, i64, i32, vp]),
        "ttt_stream_ex": (ctypes.c_int, [i32, i32, i32, vp, vp, vp, vp, vp, i64, vp, i64, vp, i64, vp, i64, i64,
                                         i64, f32, i32, i32, u32, vp, sz, vp]),
        "ttt_apply": (ctypes.c_int, [i32, i32, i32, vp, vp, vp, vp, i64, vp, i64, i64, i32, vp, sz, vp]),
        "ttt_shortconv2d": (ctypes.c_int, [vp, vp, i64, vp, i32, i32, i32, i32, i32, i32, i32, vp]),
        "ttt_stream": (ctypes.c_int, [i32, i32, i32, vp, vp, vp, vp, vp, i64, vp, i64, vp, i64, vp, i64, i64, i64,
                                      f32, i32, i32, vp, sz, vp]),
        "ttt_set_option": (ctypes.c_int, [i32, i64]),
        "ttt_profile_enable": (ctypes.c_int, [i32]),
        "ttt_profile_reset": (ctypes.c_int, []),
        "ttt_profile_read": (ctypes.c_int, [i32, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)]),
        "ttt_delta_workspace_bytes": (ctypes.c_int, [i32, i32, i32, i32, i64, i32, i32, i32, szp]),
        "ttt_delta": (ctypes.c_int, [i32, i32, i32, i32, vp, vp, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64,
                                     i64, vp, i32, f32, i32, u32, vp, sz, vp]),
        "ttt_delta_backward": (ctypes.c_int, [i32, i32, i32, i32, vp, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp,
                                              i64, vp, vp, i64, vp, i64, vp, i64, vp, vp, vp, i64, vp, i32, f32, i32,
                                              vp, sz, vp]),
        "ttt_delta_step": (ctypes.c_int, [i32, i32, i32, i32, vp, i32, vp, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64,
                                          vp, i64, i64, f32, i32, u32, vp]),
        "ttt_gated_residual": (ctypes.c_int, [i32, i32, vp, i64, vp, i64, vp, i64, vp, vp, vp, f32, vp, i64, vp, i64,
                                              i64, i32, vp]),
        "ttt_gated_residual_backward_workspace_bytes": (ctypes.c_int, [i32, i64, szp]),
        "ttt_gated_residual_backward": (ctypes.c_int, [i32, i32, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp,
                                                       vp, f32, vp, i64, vp, i64, vp, i64, vp, vp, vp, i64, i32, vp,
                                                       sz, vp]),
        "ttt_orthogonalise_workspace_bytes": (ctypes.c_int, [i32, i32, i32, i32, szp]),
        "ttt_orthogonalise": (ctypes.c_int, [i32, i32, i32, vp, i64, i64, vp, i64, i64, i32, i32, vp, sz, vp]),
        "ttt_window_attention_workspace_bytes": (ctypes.c_int, [i32, i32, i32, i64, i64] + 7 * [i32] + [szp]),
        "ttt_window_attention": (ctypes.c_int, [i32, i32, i32, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i64, vp, vp,
                                                i32, i32, i32, i32, i32, f32, i32, u32, vp, sz, vp]),
        "ttt_window_attention_backward": (ctypes.c_int, [i32, i32, i32] + 4 * [vp, i64] + [vp] + 4 * [vp, i64] +
                                          [i64, i64, vp, vp, i32, i32, i32, i32, i32, f32, i32, vp, sz, vp]),
        "ttt_window_attention_step_workspace_bytes": (ctypes.c_int, [i32, i32, i32, i64, i32, i32, szp]),
        "ttt_window_attention_step": (ctypes.c_int, [i32, i32, i32, vp, vp, i64, i64, i32, i32, vp, vp] +
                                      4 * [vp, i64] + [i64, i32, i32, i32, f32, i32, u32, vp, sz, vp]),
        "ttt_layer_norm": (ctypes.c_int, [i32, i32, vp, i64, vp, vp, f32, vp, i64, i64, i32, vp]),
        "ttt_layer_norm_backward_workspace_bytes": (ctypes.c_int, [i32, i32, i64, szp]),
        "ttt_layer_norm_backward": (ctypes.c_int, [i32, i32, vp, i64, vp, i64, vp, f32, vp, i64, vp, vp, i64, i32, vp,
                                                   sz, vp]),
        "ttt_adamw_check": (ctypes.c_int, [ctypes.POINTER(_AdamwTensor), i32, i32, i32]),
        "ttt_adamw_step": (ctypes.c_int, [ctypes.POINTER(_AdamwTensor), i32, i64, vp] + [ctypes.c_double, vp] +
                           4 * [ctypes.c_double] + [vp, i32, i32, vp, sz, vp]),
        "ttt_mfma_rate_probe": (ctypes.c_int, [i32, vp, ctypes.POINTER(ctypes.c_double)]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
    _lib = L
    return L


def _check(status: int) -> None:
    if status != 0:
        msg = load().ttt_last_error().decode(errors="replace")
        raise TTTError(f"libttt status {status}: {msg}")


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return TTT_BF16
    if t.dtype == torch.float32:
        return TTT_F32
    raise TypeError(f"token tensors must be bfloat16 or float32, got {t.dtype}")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream() -> int:
    # the raw handle of torch.cuda.current_stream(), without building its object (several us a call)
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _rows(t: torch.Tensor, name: str) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    return t.stride(0)


def _weights(w: Sequence[torch.Tensor]) -> Tuple[int, int, int]:
    w1, w3, w2 = w
    for x in w:
        if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
            raise ValueError("fast weights must be contiguous float32 GPU tensors")
    H, m, d = w1.shape
    if w3.shape != (H, m, d) or w2.shape != (H, d, m):
        raise ValueError(f"weight shapes {tuple(w1.shape)}, {tuple(w3.shape)}, {tuple(w2.shape)} do not match")
    return H, d, m


def _eta_stride(eta: torch.Tensor, H: int, n: int, device, on_gpu: bool = True, name: str = "eta") -> int:
    """Head stride of the rates: [H, >=n] with unit token stride, or [>=n] shared by every head."""
    if eta.dtype != torch.float32:
        raise ValueError(f"{name} must be float32")
    if on_gpu:
        if not eta.is_cuda or (device is not None and eta.device != torch.device(device)):
            raise ValueError(f"{name} must be on the same GPU as the tokens")
    elif eta.is_cuda:
        raise ValueError(f"{name} must be in host memory")
    if eta.dim() == 2:
        if eta.shape[0] != H or eta.shape[1] < n or (n > 1 and eta.stride(1) != 1) or eta.stride(0) < 0:
            raise ValueError(f"{name} must be [H={H}, >={n}] with unit token stride")
        return eta.stride(0)
    if eta.dim() == 1:
        if eta.shape[0] < n or (n > 1 and eta.stride(0) != 1):
            raise ValueError(f"{name} must be [>={n}] with unit stride")
        return 0
    raise ValueError(f"{name} must be [H, N] or [N]")


def _same_rows(t: torch.Tensor, like: torch.Tensor, rows: int, width: int, name: str) -> int:
    """`t` is a [rows, >=width] tensor of like's dtype and device with unit column stride;
    returns its row stride."""
    if t.dtype != like.dtype:
        raise ValueError(f"{name} must have dtype {like.dtype}, got {t.dtype}")
    if t.device != like.device:
        raise ValueError(f"{name} must be on {like.device}")
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] < width or t.stride(1) != 1:
        raise ValueError(f"{name} must be [{rows}, >={width}] with unit column stride, got {tuple(t.shape)}")
    return t.stride(0)


def _workspace(nbytes: int, device) -> Optional[torch.Tensor]:
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def set_option(option: int, value: int) -> None:
    _check(load().ttt_set_option(option, value))


def update_workspace_bytes(heads: int, d: int, m: int, n: int, dtype: torch.dtype) -> int:
    out = ctypes.c_size_t()
    code = TTT_BF16 if dtype == torch.bfloat16 else TTT_F32
    _check(load().ttt_update_workspace_bytes(heads, d, m, n, code, ctypes.byref(out)))
    return out.value


def apply_workspace_bytes(heads: int, d: int, m: int, nq: int, dtype: torch.dtype) -> int:
    out = ctypes.c_size_t()
    code = TTT_BF16 if dtype == torch.bfloat16 else TTT_F32
    _check(load().ttt_apply_workspace_bytes(heads, d, m, nq, code, ctypes.byref(out)))
    return out.value


def update(w: Sequence[torch.Tensor], k: torch.Tensor, v: torch.Tensor, eta: torch.Tensor, lr: float,
           steps: int = 1, out: Optional[Sequence[torch.Tensor]] = None, grad_out: Optional[torch.Tensor] = None,
           ns_out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
           norm_preserve: bool = False):
    """Fast-weight update; returns (W1^, W3^, W2^).  ``out`` may be ``w`` (in place).

    ``norm_preserve`` selects the norm-preserving step (flag TTT_NORM_PRESERVE).
    """
    H, d, m = _weights(w)
    if out is None:
        out = tuple(torch.empty_like(x) for x in w)
    _weights(out)
    n = k.shape[0]
    code = _dtype_code(k)
    if v.dtype != k.dtype or v.shape != k.shape or v.stride() != k.stride():
        raise ValueError("k and v must share dtype, shape and strides")
    ld = _rows(k, "k")
    if k.shape[1] < H * d:
        raise ValueError(f"k rows must hold H*d = {H * d} columns")
    ehs = _eta_stride(eta, H, n, k.device)
    for t, name in ((grad_out, "grad_out"), (ns_out, "ns_out")):
        if t is not None and (t.dtype != torch.float32 or t.numel() != 3 * H * d * m or not t.is_contiguous()
                              or t.device != k.device):
            raise ValueError(f"{name} must be a contiguous float32 tensor of 3*H*m*d elements on k's GPU")
    need = update_workspace_bytes(H, d, m, n, k.dtype)
    if workspace is None:
        workspace = _workspace(need, k.device)
    flags = NORM_PRESERVE if norm_preserve else 0
    _check(load().ttt_update_ex(H, d, m, *map(_ptr, w), *map(_ptr, out), k.data_ptr(), v.data_ptr(), ld,
                                eta.data_ptr(), ehs, n, float(lr), int(steps), code, flags, _ptr(grad_out),
                                _ptr(ns_out), _ptr(workspace), workspace.numel() if workspace is not None else 0,
                                _stream()))
    return tuple(out)


def update_noalloc(w: Sequence[torch.Tensor], k: torch.Tensor, v: torch.Tensor, eta: torch.Tensor, lr: float,
                   steps: int = 1, out: Optional[Sequence[torch.Tensor]] = None,
                   grad_out: Optional[torch.Tensor] = None, ns_out: Optional[torch.Tensor] = None,
                   norm_preserve: bool = False):
    """``update`` through the allocation-free entry point (library-owned scratch, no
    workspace).  ``out`` must be given by callers that may not allocate."""
    H, d, m = _weights(w)
    if out is None:
        out = tuple(torch.empty_like(x) for x in w)
    _weights(out)
    n = k.shape[0]
    code = _dtype_code(k)
    if v.dtype != k.dtype or v.shape != k.shape or v.stride() != k.stride():
        raise ValueError("k and v must share dtype, shape and strides")
    ld = _rows(k, "k")
    if k.shape[1] < H * d:
        raise ValueError(f"k rows must hold H*d = {H * d} columns")
    ehs = _eta_stride(eta, H, n, k.device)
    for t, name in ((grad_out, "grad_out"), (ns_out, "ns_out")):
        if t is not None and (t.dtype != torch.float32 or t.numel() != 3 * H * d * m or not t.is_contiguous()
                              or t.device != k.device):
            raise ValueError(f"{name} must be a contiguous float32 tensor of 3*H*m*d elements on k's GPU")
    flags = NORM_PRESERVE if norm_preserve else 0
    _check(load().ttt_update_noalloc(H, d, m, *map(_ptr, w), *map(_ptr, out), k.data_ptr(), v.data_ptr(), ld,
                                     eta.data_ptr(), ehs, n, float(lr), int(steps), code, flags, _ptr(grad_out),
                                     _ptr(ns_out), _stream()))
    return tuple(out)


def noalloc_scratch_bytes() -> int:
    out = ctypes.c_size_t()
    _check(load().ttt_noalloc_scratch_bytes(ctypes.byref(out)))
    return out.value


def update_host_workspace_bytes(heads: int, d: int, m: int, batch: int, ld: int, dtype: torch.dtype) -> int:
    out = ctypes.c_size_t()
    code = TTT_BF16 if dtype == torch.bfloat16 else TTT_F32
    _check(load().ttt_update_host_workspace_bytes(heads, d, m, batch, ld, code, ctypes.byref(out)))
    return out.value


def update_host(w: Sequence[torch.Tensor], k: torch.Tensor, v: torch.Tensor, eta: torch.Tensor, lr: float,
                steps: int = 1, batch: int = 65536, out: Optional[Sequence[torch.Tensor]] = None,
                grad_out: Optional[torch.Tensor] = None, ns_out: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, norm_preserve: bool = False):
    """Fast-weight update with K, V, eta in host memory (pinned for overlap), streamed in batches."""
    H, d, m = _weights(w)
    if out is None:
        out = tuple(torch.empty_like(x) for x in w)
    _weights(out)
    n = k.shape[0]
    code = _dtype_code(k)
    if k.is_cuda or v.is_cuda or eta.is_cuda:
        raise ValueError("update_host takes k, v and eta in host memory")
    if v.dtype != k.dtype or v.shape != k.shape or v.stride() != k.stride() or k.dim() != 2 or k.stride(1) != 1:
        raise ValueError("k and v must be 2-D host tensors sharing dtype, shape and strides")
    if k.shape[1] < H * d:
        raise ValueError(f"k rows must hold H*d = {H * d} columns")
    ehs = _eta_stride(eta, H, n, None, on_gpu=False)
    for t, name in ((grad_out, "grad_out"), (ns_out, "ns_out")):
        if t is not None and (t.dtype != torch.float32 or t.numel() != 3 * H * d * m or not t.is_contiguous()
                              or t.device != w[0].device):
            raise ValueError(f"{name} must be a contiguous float32 tensor of 3*H*m*d elements on the weights' GPU")
    ld = k.stride(0)
    need = update_host_workspace_bytes(H, d, m, batch, ld, k.dtype)
    if workspace is None:
        workspace = _workspace(need, w[0].device)
    flags = NORM_PRESERVE if norm_preserve else 0
    _check(load().ttt_update_host(H, d, m, *map(_ptr, w), *map(_ptr, out), k.data_ptr(), v.data_ptr(), ld,
                                  eta.data_ptr(), ehs, n, batch, float(lr), int(steps), code, flags, _ptr(grad_out),
                                  _ptr(ns_out), _ptr(workspace), workspace.numel() if workspace is not None else 0,
                                  _stream()))
    return tuple(out)


def apply(w: Sequence[torch.Tensor], q: torch.Tensor, out: Optional[torch.Tensor] = None,
          workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """o_i = f_W(q_i) for every row of q."""
    H, d, m = _weights(w)
    code = _dtype_code(q)
    ldq = _rows(q, "q")
    if q.shape[1] < H * d:
        raise ValueError(f"q rows must hold H*d = {H * d} columns")
    if out is None:
        out = torch.empty((q.shape[0], H * d), dtype=q.dtype, device=q.device)
    ldo = _same_rows(out, q, q.shape[0], H * d, "out")
    need = apply_workspace_bytes(H, d, m, q.shape[0], q.dtype)
    if workspace is None:
        workspace = _workspace(need, q.device)
    _check(load().ttt_apply(H, d, m, *map(_ptr, w), q.data_ptr(), ldq, out.data_ptr(), ldo, q.shape[0], code,
                            _ptr(workspace), workspace.numel() if workspace is not None else 0, _stream()))
    return out


def shortconv2d(v: torch.Tensor, wconv: torch.Tensor, frames: int, tokens_per_frame: int, n_special: int,
                grid_h: int, grid_w: int, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """V' = ShortConv2D(V) over each frame's patch grid (depthwise 3x3, zero padding)."""
    code = _dtype_code(v)
    ld = _rows(v, "v")
    C = v.shape[1]
    if wconv.dtype != torch.float32 or tuple(wconv.shape) != (C, 3, 3) or not wconv.is_contiguous():
        raise ValueError("wconv must be contiguous float32 [C, 3, 3]")
    if out is None:
        out = torch.empty_like(v)
    if out.stride() != v.stride():
        raise ValueError("out must have the same strides as v")
    _check(load().ttt_shortconv2d(v.data_ptr(), out.data_ptr(), ld, wconv.data_ptr(), frames, tokens_per_frame,
                                  n_special, grid_h, grid_w, C, code, _stream()))
    return out


def stream_workspace_bytes(heads: int, d: int, m: int, chunk: int, dtype: torch.dtype) -> int:
    out = ctypes.c_size_t()
    code = TTT_BF16 if dtype == torch.bfloat16 else TTT_F32
    _check(load().ttt_stream_workspace_bytes(heads, d, m, chunk, code, ctypes.byref(out)))
    return out.value


def stream(w: Sequence[torch.Tensor], k: torch.Tensor, v: torch.Tensor, eta: torch.Tensor, q: torch.Tensor,
           lr: float, steps: int, chunk: int, out: Optional[torch.Tensor] = None,
           workspace: Optional[torch.Tensor] = None, norm_preserve: bool = False) -> torch.Tensor:
    """Chunked causal pass: per chunk apply then update; ``w`` is updated in place."""
    H, d, m = _weights(w)
    code = _dtype_code(k)
    n = k.shape[0]
    ld = _rows(k, "k")
    if k.shape[1] < H * d:
        raise ValueError(f"k rows must hold H*d = {H * d} columns")
    if v.stride() != k.stride():
        raise ValueError("k and v must share strides")
    _same_rows(v, k, n, H * d, "v")
    ldq = _same_rows(q, k, n, H * d, "q")
    if out is None:
        out = torch.empty((n, H * d), dtype=q.dtype, device=q.device)
    ldo = _same_rows(out, k, n, H * d, "out")
    ehs = _eta_stride(eta, H, n, k.device)
    need = stream_workspace_bytes(H, d, m, chunk, k.dtype)
    if workspace is None:
        workspace = _workspace(need, k.device)
    flags = NORM_PRESERVE if norm_preserve else 0
    _check(load().ttt_stream_ex(H, d, m, *map(_ptr, w), k.data_ptr(), v.data_ptr(), ld, eta.data_ptr(), ehs,
                                q.data_ptr(), ldq, out.data_ptr(), ldo, n, chunk, float(lr), int(steps), code, flags,
                                _ptr(workspace), workspace.numel() if workspace is not None else 0, _stream()))
    return out


def output_gate(o: torch.Tensor, wg: torch.Tensor, gamma: torch.Tensor, eps: float,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """o_i = RMSNorm(o'_i) * SiLU(W_g o'_i) over rows of C = wg.shape[0] channels."""
    code = _dtype_code(o)
    C = wg.shape[0]
    if wg.dtype != o.dtype or tuple(wg.shape) != (C, C) or not wg.is_contiguous() or not wg.is_cuda:
        raise ValueError("wg must be a contiguous [C, C] GPU tensor of o's dtype")
    if gamma.dtype != torch.float32 or tuple(gamma.shape) != (C,) or not gamma.is_contiguous() or not gamma.is_cuda:
        raise ValueError("gamma must be a contiguous float32 [C] GPU tensor")
    ldi = _rows(o, "o")
    if o.shape[1] < C:
        raise ValueError(f"o rows must hold C = {C} columns")
    if wg.device != o.device or gamma.device != o.device:
        raise ValueError("wg and gamma must be on o's GPU")
    if out is None:
        out = torch.empty((o.shape[0], C), dtype=o.dtype, device=o.device)
    ldo = _same_rows(out, o, o.shape[0], C, "out")
    _check(load().ttt_output_gate(C, o.data_ptr(), ldi, wg.data_ptr(), gamma.data_ptr(), float(eps), out.data_ptr(),
                                  ldo, o.shape[0], code, _stream()))
    return out


# ------------------------------------------------------------------ gated delta rule
# A call of one token takes a few microseconds on the GPU: the checks below ask each tensor for few
# things, in one expression where all is well, and look for what is wrong only where it is not.
def _gpu(t: torch.Tensor, name: str) -> int:
    """The current GPU's index; `t` must live there (the library launches on its current stream)."""
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name} must be on the current GPU, got {t.device}")
    return dev


def _row(t: torch.Tensor, dtype: torch.dtype, dev: int, n: int, width: int, name: str) -> int:
    """`t` is [n, >=width] rows of `dtype` on GPU `dev` with unit column stride; returns its row stride."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 2 and shape[0] == n and shape[1] >= width and stride[1] == 1 and t.dtype == dtype \
            and t.get_device() == dev:
        return stride[0]
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be [{n}, >={width}] with unit column stride, got {tuple(shape)}")


def _rate(t: torch.Tensor, H: int, n: int, dev: int, name: str) -> int:
    """Head stride of a rate tensor (as _eta_stride)."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 2 and shape[0] == H and shape[1] >= n and stride[1] == 1 and t.dtype == torch.float32 \
            and t.get_device() == dev:
        return stride[0]
    return _eta_stride(t, H, n, torch.device("cuda", dev), name=name)


# (ctypes takes the low 32 bits of a larger number, without a word)
_MAX32 = (1 << 31) - 1


def _int32(x: int, name: str) -> int:
    if not -_MAX32 <= x <= _MAX32:
        raise ValueError(f"{name} must be less than 2^31, got {x}")
    return int(x)


def _bytes(workspace: torch.Tensor, dev: int) -> int:
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on cuda:{dev}")
    return workspace.numel() * workspace.element_size()


def _states(w: torch.Tensor, like: Optional[torch.Tensor], name: str) -> None:
    if w.dtype != torch.float32 or w.dim() != 4 or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor [sequences, heads, dv, dk]")
    if like is not None and (w.shape != like.shape or w.get_device() != like.get_device()):
        raise ValueError(f"{name} must have w's shape and device")


def _delta_args(w, q, k, v, beta, decay, key_heads):
    """Checks shared by the delta-rule calls."""
    _states(w, None, "w")
    dev = _gpu(w, "w")
    S, H, dv, dk = w.shape
    Hk = H if key_heads is None else int(key_heads)
    code = _dtype_code(q)
    dtype = q.dtype
    if q.dim() != 2:
        raise ValueError("q must be a 2-D tensor of token rows")
    n = q.shape[0]
    return (dev, S, H, Hk, dv, dk, n, code, _row(q, dtype, dev, n, Hk * dk, "q"), _row(k, dtype, dev, n, Hk * dk, "k"),
            _row(v, dtype, dev, n, H * dv, "v"), _rate(beta, H, n, dev, "beta"),
            0 if decay is None else _rate(decay, H, n, dev, "decay"))


def _offsets(cu, sequences: int, dev: int) -> None:
    if cu is None:
        if sequences != 1:
            raise ValueError(f"w holds {sequences} states: cu_seqlens is needed for more than one sequence")
    elif cu.dtype != torch.int32 or tuple(cu.shape) != (sequences + 1,) or not cu.is_contiguous() \
            or cu.get_device() != dev:
        raise ValueError(f"cu_seqlens must be a contiguous int32 tensor [{sequences + 1}] on cuda:{dev}")


def delta_workspace_bytes(heads: int, key_heads: int, dk: int, dv: int, n: int, sequences: int, dtype: torch.dtype,
                          backward: bool = False) -> int:
    out = ctypes.c_size_t()
    code = TTT_BF16 if dtype == torch.bfloat16 else TTT_F32
    _check(load().ttt_delta_workspace_bytes(heads, key_heads, dk, dv, n, sequences, code, int(backward),
                                            ctypes.byref(out)))
    return out.value


def delta(w: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor,
          decay: Optional[torch.Tensor] = None, *, key_heads: Optional[int] = None,
          cu_seqlens: Optional[torch.Tensor] = None, scale: Optional[float] = None,
          out: Optional[torch.Tensor] = None, w_out: Optional[torch.Tensor] = None,
          workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Gated delta rule over packed sequences; returns (o, final states).

    w [sequences, H, dv, dk] float32 starting states; q, k rows of key_heads * dk, v rows of H * dv columns;
    beta and decay (log decay, None: no decay) [H, >=n] or shared [>=n].  ``w_out`` may be ``w`` (in place).
    Rows outside the sequences stay as they are in a given ``out`` and are zero in a new one.
    """
    dev, S, H, Hk, dv, dk, n, code, ldq, ldk, ldv, bhs, dhs = _delta_args(w, q, k, v, beta, decay, key_heads)
    _offsets(cu_seqlens, S, dev)
    flags, ldo = 0, H * dv
    if out is None:
        out = q.new_empty((n, H * dv))
        flags = DELTA_ZERO_UNUSED
    else:
        ldo = _row(out, q.dtype, dev, n, H * dv, "out")
    if w_out is None:
        w_out = torch.empty_like(w)
    else:
        _states(w_out, w, "w_out")
    if workspace is None:
        workspace = _workspace(delta_workspace_bytes(H, Hk, dk, dv, n, S, q.dtype), w.device)
    _check(load().ttt_delta(H, Hk, dk, dv, w.data_ptr(), w_out.data_ptr(), q.data_ptr(), ldq, k.data_ptr(), ldk,
                            v.data_ptr(), ldv, beta.data_ptr(), bhs, _ptr(decay), dhs, out.data_ptr(), ldo, n,
                            _ptr(cu_seqlens), S, 1.0 if scale is None else float(scale), code, flags,
                            workspace.data_ptr(), _bytes(workspace, dev), _stream()))
    return out, w_out


def delta_backward(w: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor,
                   decay: Optional[torch.Tensor], grad_o: torch.Tensor, grad_w_out: Optional[torch.Tensor] = None, *,
                   key_heads: Optional[int] = None, cu_seqlens: Optional[torch.Tensor] = None,
                   scale: Optional[float] = None, out: Optional[Sequence[torch.Tensor]] = None,
                   workspace: Optional[torch.Tensor] = None):
    """Gradients of ``delta``: (grad_q, grad_k, grad_v, grad_beta, grad_decay, grad_w).

    ``out`` gives (grad_q, grad_k, grad_v) rows to write to (slices of one buffer, say).  grad_beta and
    grad_decay are [H, n], or [n] for shared rates; grad_decay is None without decay.
    """
    dev, S, H, Hk, dv, dk, n, code, ldq, ldk, ldv, bhs, dhs = _delta_args(w, q, k, v, beta, decay, key_heads)
    _offsets(cu_seqlens, S, dev)
    dtype = q.dtype
    ldgo = _row(grad_o, dtype, dev, n, H * dv, "grad_o")
    if grad_w_out is not None:
        _states(grad_w_out, w, "grad_w_out")
    if out is None:
        out = tuple(torch.empty((n, x), dtype=dtype, device=q.device) for x in (Hk * dk, Hk * dk, H * dv))
    gq, gk, gv = out
    # a 2-D rate broadcast over heads (stride 0) still gets a gradient for each head
    if beta.dim() == 2 and bhs == 0:
        beta, bhs = beta[:, :n].contiguous(), n
    if decay is not None and decay.dim() == 2 and dhs == 0:
        decay, dhs = decay[:, :n].contiguous(), n
    gb = torch.empty((H, n) if beta.dim() == 2 else (n,), dtype=torch.float32, device=w.device)
    gd = None if decay is None else torch.empty((H, n) if decay.dim() == 2 else (n,), dtype=torch.float32,
                                                device=w.device)
    gw = torch.empty_like(w)
    if workspace is None:
        workspace = _workspace(delta_workspace_bytes(H, Hk, dk, dv, n, S, dtype, True), w.device)
    _check(load().ttt_delta_backward(H, Hk, dk, dv, w.data_ptr(), q.data_ptr(), ldq, k.data_ptr(), ldk,
                                     v.data_ptr(), ldv, beta.data_ptr(), bhs, _ptr(decay), dhs, grad_o.data_ptr(),
                                     ldgo, _ptr(grad_w_out), gq.data_ptr(), _row(gq, dtype, dev, n, Hk * dk, "grad_q"),
                                     gk.data_ptr(), _row(gk, dtype, dev, n, Hk * dk, "grad_k"), gv.data_ptr(),
                                     _row(gv, dtype, dev, n, H * dv, "grad_v"), gb.data_ptr(), _ptr(gd),
                                     gw.data_ptr(), n, _ptr(cu_seqlens), S, 1.0 if scale is None else float(scale),
                                     code, workspace.data_ptr(), _bytes(workspace, dev), _stream()))
    return gq, gk, gv, gb, gd, gw


def delta_step(w: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor,
               decay: Optional[torch.Tensor] = None, *, slots: Optional[torch.Tensor] = None,
               key_heads: Optional[int] = None, scale: Optional[float] = None,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token for each row, its state in the pool ``w`` [pool, H, dv, dk] updated in place; returns o.

    Row i uses state ``slots[i]`` (int32; None: state i).  Slots outside the pool are padding: such rows
    stay as they are in a given ``out`` and are zero in a new one.  Rows of one state apply in row order.
    """
    dev, S, H, Hk, dv, dk, n, code, ldq, ldk, ldv, bhs, dhs = _delta_args(w, q, k, v, beta, decay, key_heads)
    if slots is not None and (slots.dtype != torch.int32 or slots.shape != (n,) or not slots.is_contiguous()
                              or slots.get_device() != dev):
        raise ValueError(f"slots must be a contiguous int32 tensor [{n}] on cuda:{dev}")
    flags, ldo = 0, H * dv
    if out is None:
        out = q.new_empty((n, H * dv))
        flags = DELTA_ZERO_UNUSED
    else:
        ldo = _row(out, q.dtype, dev, n, H * dv, "out")
    _check(load().ttt_delta_step(H, Hk, dk, dv, w.data_ptr(), S, _ptr(slots), q.data_ptr(), ldq, k.data_ptr(), ldk,
                                 v.data_ptr(), ldv, beta.data_ptr(), bhs, _ptr(decay), dhs, out.data_ptr(), ldo, n,
                                 1.0 if scale is None else float(scale), code, flags, _stream()))
    return out


# ------------------------------------------------------------------ gated residual tail
def _channel(t: Optional[torch.Tensor], C: int, dev: int, name: str) -> Optional[int]:
    if t is None:
        return None
    if t.dtype != torch.float32 or t.shape != (C,) or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous float32 [{C}] tensor on cuda:{dev}")
    return t.data_ptr()


def gated_residual(x: torch.Tensor, o: torch.Tensor, z: Optional[torch.Tensor] = None,
                   gamma: Optional[torch.Tensor] = None, alpha: Optional[torch.Tensor] = None,
                   gamma_next: Optional[torch.Tensor] = None, eps: float = 1e-6, *, norm_width: Optional[int] = None,
                   out: Optional[torch.Tensor] = None, h_out: Optional[torch.Tensor] = None):
    """y = x + alpha * RMSNorm(o; gamma) * SiLU(z), h = RMSNorm(y; gamma_next); returns (y, h).

    The first norm runs over groups of ``norm_width`` channels (default: the row).  z None: no gate;
    gamma or alpha None: 1; gamma_next None: h is None.  ``out`` may be ``x`` (in place).
    """
    code, dtype, dev = _dtype_code(x), x.dtype, _gpu(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be a 2-D tensor of rows")
    n, C = x.shape
    ldx, ldo = _row(x, dtype, dev, n, C, "x"), _row(o, dtype, dev, n, C, "o")
    ldz = 0 if z is None else _row(z, dtype, dev, n, C, "z")
    gamma, alpha = _channel(gamma, C, dev, "gamma"), _channel(alpha, C, dev, "alpha")
    gamma_next = _channel(gamma_next, C, dev, "gamma_next")
    ldy = ldh = C
    if out is None:
        out = x.new_empty((n, C))
    else:
        ldy = _row(out, dtype, dev, n, C, "out")
    if h_out is not None:
        if gamma_next is None:
            raise ValueError("h_out needs gamma_next")
        ldh = _row(h_out, dtype, dev, n, C, "h_out")
    elif gamma_next is not None:
        h_out = x.new_empty((n, C))
    w = C if norm_width is None else _int32(norm_width, "norm_width")
    _check(load().ttt_gated_residual(C, w, x.data_ptr(), ldx, o.data_ptr(), ldo, _ptr(z), ldz, gamma, alpha,
                                     gamma_next, float(eps), out.data_ptr(), ldy, _ptr(h_out), ldh, n, code, _stream()))
    return out, h_out


def gated_residual_backward_workspace_bytes(channels: int, n: int) -> int:
    out = ctypes.c_size_t()
    _check(load().ttt_gated_residual_backward_workspace_bytes(channels, n, ctypes.byref(out)))
    return out.value


def gated_residual_backward(grad_y: Optional[torch.Tensor], grad_h: Optional[torch.Tensor], y: torch.Tensor,
                            o: torch.Tensor, z: Optional[torch.Tensor] = None, gamma: Optional[torch.Tensor] = None,
                            alpha: Optional[torch.Tensor] = None, gamma_next: Optional[torch.Tensor] = None,
                            eps: float = 1e-6, *, norm_width: Optional[int] = None,
                            workspace: Optional[torch.Tensor] = None):
    """Gradients of ``gated_residual``: (grad_x, grad_o, grad_z, grad_gamma, grad_alpha, grad_gamma_next).

    ``y`` is the forward's output.  grad_y or grad_h None: zero.  The gradients of what was not given
    are None.
    """
    code, dtype, dev = _dtype_code(y), y.dtype, _gpu(y, "y")
    if y.dim() != 2:
        raise ValueError("y must be a 2-D tensor of rows")
    n, C = y.shape
    ld = lambda t, name: 0 if t is None else _row(t, dtype, dev, n, C, name)
    ldgy, ldgh, ldy = ld(grad_y, "grad_y"), ld(grad_h, "grad_h"), ld(y, "y")
    ldo, ldz = _row(o, dtype, dev, n, C, "o"), ld(z, "z")
    w = C if norm_width is None else _int32(norm_width, "norm_width")
    given = gamma is not None, alpha is not None, gamma_next is not None
    gamma, alpha = _channel(gamma, C, dev, "gamma"), _channel(alpha, C, dev, "alpha")
    gamma_next = _channel(gamma_next, C, dev, "gamma_next")
    gx, go = torch.empty((n, C), dtype=dtype, device=y.device), torch.empty((n, C), dtype=dtype, device=y.device)
    gz = None if z is None else torch.empty((n, C), dtype=dtype, device=y.device)
    gg, ga, gn = (torch.empty(C, dtype=torch.float32, device=y.device) if g else None for g in given)
    if workspace is None:
        workspace = _workspace(gated_residual_backward_workspace_bytes(C, n), y.device)
    _check(load().ttt_gated_residual_backward(
        C, w, _ptr(grad_y), ldgy, _ptr(grad_h), ldgh, y.data_ptr(), ldy, o.data_ptr(), ldo, _ptr(z), ldz,
        gamma, alpha, gamma_next, float(eps), gx.data_ptr(), C, go.data_ptr(), C, _ptr(gz), C, _ptr(gg), _ptr(ga),
        _ptr(gn), n, code, workspace.data_ptr(), _bytes(workspace, dev), _stream()))
    return gx, go, gz, gg, ga, gn


# ------------------------------------------------------------------ orthogonalisation
def orthogonalise_workspace_bytes(rows: int, cols: int, batch: int, dtype: torch.dtype) -> int:
    out = ctypes.c_size_t()
    code = TTT_BF16 if dtype == torch.bfloat16 else TTT_F32
    _check(load().ttt_orthogonalise_workspace_bytes(rows, cols, batch, code, ctypes.byref(out)))
    return out.value


def orthogonalise(g: torch.Tensor, steps: int = 5, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Muon's Newton-Schulz orthogonalisation of g [rows, cols] or of every matrix of g [batch, rows, cols].

    ``out`` may be ``g`` (in place).
    """
    code, dev = _dtype_code(g), _gpu(g, "g")
    if out is None:
        out = torch.empty(g.shape, dtype=g.dtype, device=g.device)
    for t, name in ((g, "g"), (out, "out")):
        if t.dim() not in (2, 3) or t.stride(-1) != 1 or t.dtype != g.dtype or t.shape != g.shape \
                or t.get_device() != dev:
            raise ValueError(f"{name} must be [rows, cols] or [batch, rows, cols] of one dtype and device with unit "
                             f"column stride")
    B, R, C = (1, *g.shape) if g.dim() == 2 else g.shape
    bs = lambda t: t.stride(0) if t.dim() == 3 else 0
    if workspace is None:
        workspace = _workspace(orthogonalise_workspace_bytes(R, C, B, g.dtype), g.device)
    _check(load().ttt_orthogonalise(R, C, B, g.data_ptr(), g.stride(-2), bs(g), out.data_ptr(), out.stride(-2), bs(out),
                                    int(steps), code, _ptr(workspace),
                                    0 if workspace is None else _bytes(workspace, dev), _stream()))
    return out


# ------------------------------------------------------------------ windowed attention
def _limit(x: Optional[int], name: str) -> int:
    if x is None:
        return -1
    if x < 0:
        raise ValueError(f"{name} must be >= 0, or None for no limit")
    return int(x) if x <= _MAX32 else -1                # (no position is as far as 2^31 blocks)


def _sinks(x: int) -> int:
    return max(-1, min(int(x), _MAX32))                 # (2^31 - 1: all keys; -1 is refused)


def _heads(q: torch.Tensor, heads: int, key_heads: Optional[int]) -> Tuple[int, int, int]:
    """(heads, key_heads, d) of query rows."""
    if q.dim() != 2:
        raise ValueError("q must be a 2-D tensor of token rows")
    H = int(heads)
    if H < 1 or q.shape[1] % H != 0:
        raise ValueError(f"q rows of {q.shape[1]} columns do not hold {heads} heads")
    return H, H if key_heads is None else int(key_heads), q.shape[1] // H


def _attention_args(q, k, v, heads, key_heads, block, before, after, sinks, scale, cu, cu_k):
    """Checks shared by windowed attention and its gradient."""
    dev, dtype, code = _gpu(q, "q"), q.dtype, _dtype_code(q)
    H, Hk, d = _heads(q, heads, key_heads)
    nq, nk = q.shape[0], k.shape[0]
    ld = (_row(q, dtype, dev, nq, H * d, "q"), _row(k, dtype, dev, nk, Hk * d, "k"), _row(v, dtype, dev, nk, Hk * d, "v"))
    S = 1
    if cu is not None:
        if cu.dim() != 1 or cu.shape[0] < 2 or cu.dtype != torch.int32 or not cu.is_contiguous() or cu.get_device() != dev:
            raise ValueError(f"cu_seqlens must be a contiguous int32 tensor [sequences + 1] on cuda:{dev}")
        S = cu.shape[0] - 1
    if cu_k is not None and (cu is None or cu_k.shape != cu.shape or cu_k.dtype != torch.int32
                             or not cu_k.is_contiguous() or cu_k.get_device() != dev):
        raise ValueError("cu_seqlens_k must be a contiguous int32 tensor like cu_seqlens")
    mask = (_int32(block, "block"), _limit(before, "before"), _limit(after, "after"), _sinks(sinks))
    return dev, dtype, code, H, Hk, d, nq, nk, ld, S, mask, d ** -0.5 if scale is None else float(scale)


def window_attention_workspace_bytes(heads: int, key_heads: int, d: int, nq: int, nk: int, sequences: int, block: int,
                                     before: Optional[int], after: Optional[int], sinks: int, dtype: torch.dtype,
                                     backward: bool = False) -> int:
    out = ctypes.c_size_t()
    code = TTT_BF16 if dtype == torch.bfloat16 else TTT_F32
    _check(load().ttt_window_attention_workspace_bytes(heads, key_heads, d, nq, nk, sequences, _int32(block, "block"),
                                                       _limit(before, "before"), _limit(after, "after"), _sinks(sinks),
                                                       code, int(backward), ctypes.byref(out)))
    return out.value


# (functions of the sizes alone: a call of a few tokens takes less than asking the library takes)
@functools.lru_cache(maxsize=4096)
def _attention_bytes(*sizes: int) -> int:
    out = ctypes.c_size_t()
    _check(load().ttt_window_attention_workspace_bytes(*sizes, ctypes.byref(out)))
    return out.value


@functools.lru_cache(maxsize=4096)
def _attention_step_bytes(*sizes: int) -> int:
    out = ctypes.c_size_t()
    _check(load().ttt_window_attention_step_workspace_bytes(*sizes, ctypes.byref(out)))
    return out.value


def window_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, heads: int, key_heads: Optional[int] = None,
                     block: int = 1, before: Optional[int] = None, after: Optional[int] = 0, sinks: int = 0,
                     scale: Optional[float] = None, cu_seqlens: Optional[torch.Tensor] = None,
                     cu_seqlens_k: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                     lse_out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Softmax attention over packed sequences within a window of blocks; returns (o, lse).

    q rows of heads * d columns, k and v rows of key_heads * d.  A query of block b (``block`` tokens each; the queries
    are the last rows of their sequence's keys) sees the keys of blocks b - before .. b + after (None: no limit) and,
    of those before, the first ``sinks``: before = after = 0 is attention inside a frame, block = 1 a causal window of
    tokens.  scale None: d ** -0.5.  lse [heads, nq] float32.  Rows outside the sequences stay as they are in a given
    ``out`` and are zero in a new one; their lse is -inf.
    """
    dev, dtype, code, H, Hk, d, nq, nk, ld, S, mask, scale = _attention_args(
        q, k, v, heads, key_heads, block, before, after, sinks, scale, cu_seqlens, cu_seqlens_k)
    flags, ldo = 0, H * d
    if out is None:
        out = q.new_empty((nq, H * d))
        flags = ATTENTION_ZERO_UNUSED
    else:
        ldo = _row(out, dtype, dev, nq, H * d, "out")
    if lse_out is None:
        lse_out = q.new_empty((H, nq), dtype=torch.float32)
    elif lse_out.dtype != torch.float32 or lse_out.shape != (H, nq) or not lse_out.is_contiguous() or lse_out.get_device() != dev:
        raise ValueError(f"lse_out must be a contiguous float32 tensor [{H}, {nq}] on cuda:{dev}")
    if workspace is None:
        workspace = q.new_empty((_attention_bytes(H, Hk, d, nq, nk, S, *mask, code, 0),), dtype=torch.uint8)
    _check(load().ttt_window_attention(H, Hk, d, q.data_ptr(), ld[0], k.data_ptr(), ld[1], v.data_ptr(), ld[2],
                                       out.data_ptr(), ldo, lse_out.data_ptr(), nq, nk, _ptr(cu_seqlens),
                                       _ptr(cu_seqlens_k), S, *mask, scale, code, flags, workspace.data_ptr(),
                                       _bytes(workspace, dev), _stream()))
    return out, lse_out


def window_attention_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
                              grad_o: torch.Tensor, *, heads: int, key_heads: Optional[int] = None, block: int = 1,
                              before: Optional[int] = None, after: Optional[int] = 0, sinks: int = 0,
                              scale: Optional[float] = None, cu_seqlens: Optional[torch.Tensor] = None,
                              cu_seqlens_k: Optional[torch.Tensor] = None,
                              out: Optional[Sequence[torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None):
    """Gradients (grad_q, grad_k, grad_v) of ``window_attention``, from its outputs o and lse.

    ``out`` gives the rows to write to (slices of one buffer, say).
    """
    dev, dtype, code, H, Hk, d, nq, nk, ld, S, mask, scale = _attention_args(
        q, k, v, heads, key_heads, block, before, after, sinks, scale, cu_seqlens, cu_seqlens_k)
    ldo, ldgo = _row(o, dtype, dev, nq, H * d, "o"), _row(grad_o, dtype, dev, nq, H * d, "grad_o")
    if lse.dtype != torch.float32 or lse.shape != (H, nq) or not lse.is_contiguous() or lse.get_device() != dev:
        raise ValueError(f"lse must be a contiguous float32 tensor [{H}, {nq}] on cuda:{dev}")
    if out is None:
        out = q.new_empty((nq, H * d)), q.new_empty((nk, Hk * d)), q.new_empty((nk, Hk * d))
    gq, gk, gv = out
    if workspace is None:
        workspace = q.new_empty((_attention_bytes(H, Hk, d, nq, nk, S, *mask, code, 1),), dtype=torch.uint8)
    _check(load().ttt_window_attention_backward(
        H, Hk, d, q.data_ptr(), ld[0], k.data_ptr(), ld[1], v.data_ptr(), ld[2], o.data_ptr(), ldo, lse.data_ptr(),
        grad_o.data_ptr(), ldgo, gq.data_ptr(), _row(gq, dtype, dev, nq, H * d, "grad_q"), gk.data_ptr(),
        _row(gk, dtype, dev, nk, Hk * d, "grad_k"), gv.data_ptr(), _row(gv, dtype, dev, nk, Hk * d, "grad_v"), nq, nk,
        _ptr(cu_seqlens), _ptr(cu_seqlens_k), S, *mask, scale, code, workspace.data_ptr(), _bytes(workspace, dev),
        _stream()))
    return gq, gk, gv


def window_attention_step(k_cache: torch.Tensor, v_cache: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                          v: torch.Tensor, positions: torch.Tensor, *, heads: int, key_heads: Optional[int] = None,
                          slots: Optional[torch.Tensor] = None, block: int = 1, before: Optional[int] = None,
                          sinks: int = 0, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token for each row over rolling caches [pool, capacity, key_heads * d], which take its k and v; returns o.

    Row i has cache ``slots[i]`` (int32; None: cache i) and its token position ``positions[i]`` (int32).  Position x
    of a sequence stands in row x of its cache (x < sinks) or sinks + (x - sinks) % (capacity - sinks).  Slots outside
    the pool and negative positions are padding: such rows stay as they are in a given ``out`` and are zero in a new
    one.  The rows of a call read the caches as they were before it.
    """
    dev, dtype, code = _gpu(q, "q"), q.dtype, _dtype_code(q)
    H, Hk, d = _heads(q, heads, key_heads)
    n = q.shape[0]
    ldq, ldk, ldv = (_row(q, dtype, dev, n, H * d, "q"), _row(k, dtype, dev, n, Hk * d, "k"),
                     _row(v, dtype, dev, n, Hk * d, "v"))
    shape, stride = k_cache.shape, k_cache.stride()
    if len(shape) != 3 or shape[2] < Hk * d or stride[2] != 1 or stride[0] < 0 or stride[1] < 0 or v_cache.shape != shape \
            or v_cache.stride() != stride or k_cache.dtype != dtype or v_cache.dtype != dtype \
            or k_cache.get_device() != dev or v_cache.get_device() != dev:
        raise ValueError(f"k_cache and v_cache must be [pool, capacity, >={Hk * d}] {dtype} tensors of the same shape "
                         f"and strides, unit column stride, on cuda:{dev}")
    if positions.dtype != torch.int32 or positions.shape != (n,) or not positions.is_contiguous() \
            or positions.get_device() != dev:
        raise ValueError(f"positions must be a contiguous int32 tensor [{n}] on cuda:{dev}")
    if slots is not None and (slots.dtype != torch.int32 or slots.shape != (n,) or not slots.is_contiguous()
                              or slots.get_device() != dev):
        raise ValueError(f"slots must be a contiguous int32 tensor [{n}] on cuda:{dev}")
    flags, ldo = 0, H * d
    if out is None:
        out = q.new_empty((n, H * d))
        flags = ATTENTION_ZERO_UNUSED
    else:
        ldo = _row(out, dtype, dev, n, H * d, "out")
    if workspace is None:
        workspace = q.new_empty((_attention_step_bytes(H, Hk, d, n, shape[1], code),), dtype=torch.uint8)
    _check(load().ttt_window_attention_step(
        H, Hk, d, k_cache.data_ptr(), v_cache.data_ptr(), stride[1], stride[0], shape[0], shape[1], _ptr(slots),
        positions.data_ptr(), q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, out.data_ptr(), ldo, n,
        _int32(block, "block"), _limit(before, "before"), _sinks(sinks), d ** -0.5 if scale is None else float(scale), code, flags,
        workspace.data_ptr(), _bytes(workspace, dev), _stream()))
    return out


# ------------------------------------------------------------------ layer norm
def layer_norm(x: torch.Tensor, gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
               eps: float = 1e-6, *, norm_width: Optional[int] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """gamma * (x - mean) / sqrt(var + eps) + beta over groups of ``norm_width`` columns (default: the row).

    gamma, beta [norm_width] float32, shared by the groups (None: 1, 0).  ``out`` may be ``x`` (in place).
    """
    code, dtype, dev = _dtype_code(x), x.dtype, _gpu(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be a 2-D tensor of rows")
    n, C = x.shape
    w = C if norm_width is None else _int32(norm_width, "norm_width")
    ldx = _row(x, dtype, dev, n, C, "x")
    gamma, beta = _channel(gamma, w, dev, "gamma"), _channel(beta, w, dev, "beta")
    if out is None:
        ldy = -(-C // 8) * 8                            # rows begin on 16 bytes
        out = x.new_empty((n, C)) if ldy == C else x.new_empty((n, ldy))[:, :C]
    else:
        ldy = _row(out, dtype, dev, n, C, "out")
    _check(load().ttt_layer_norm(C, w, x.data_ptr(), ldx, gamma, beta, float(eps), out.data_ptr(), ldy, n, code,
                                 _stream()))
    return out


@functools.lru_cache(maxsize=4096)
def _norm_backward_bytes(*sizes: int) -> int:
    out = ctypes.c_size_t()
    _check(load().ttt_layer_norm_backward_workspace_bytes(*sizes, ctypes.byref(out)))
    return out.value


def layer_norm_backward(grad_y: torch.Tensor, x: torch.Tensor, gamma: Optional[torch.Tensor] = None, eps: float = 1e-6,
                        *, norm_width: Optional[int] = None, out: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None):
    """Gradients (grad_x, grad_gamma, grad_beta) of ``layer_norm``.  ``out`` (grad_x) may be ``grad_y`` (in place)."""
    code, dtype, dev = _dtype_code(x), x.dtype, _gpu(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be a 2-D tensor of rows")
    n, C = x.shape
    w = C if norm_width is None else _int32(norm_width, "norm_width")
    ldx, ldg = _row(x, dtype, dev, n, C, "x"), _row(grad_y, dtype, dev, n, C, "grad_y")
    gamma = _channel(gamma, w, dev, "gamma")
    if out is None:
        ldo = -(-C // 8) * 8
        out = x.new_empty((n, C)) if ldo == C else x.new_empty((n, ldo))[:, :C]
    else:
        ldo = _row(out, dtype, dev, n, C, "out")
    if workspace is None:
        workspace = x.new_empty((_norm_backward_bytes(C, w, n),), dtype=torch.uint8)
    ggamma, gbeta = x.new_empty((w,), dtype=torch.float32), x.new_empty((w,), dtype=torch.float32)
    _check(load().ttt_layer_norm_backward(C, w, grad_y.data_ptr(), ldg, x.data_ptr(), ldx, gamma, float(eps),
                                          out.data_ptr(), ldo, ggamma.data_ptr(), gbeta.data_ptr(), n, code,
                                          workspace.data_ptr(), _bytes(workspace, dev), _stream()))
    return out, ggamma, gbeta


# ------------------------------------------------------------------ AdamW
class AdamwTensors:
    """The tensors of ``adamw_step``: made once by ``adamw_tensors``, it keeps their memory alive."""

    def __init__(self, table, sizes, dtype, bits, dev, lists, weights):
        self.table, self.sizes, self.dtype, self.bits, self.dev = table, sizes, dtype, bits, dev
        # (views of their own: a tensor whose ``data`` is set anew lets go of the memory that the table names)
        self.held = [t.detach() for x in lists for t in x]
        self.weights = weights                          # params and masters, which are looked at in every step
        self.at = [t.data_ptr() for t in weights]


def adamw_tensors(params: Sequence[torch.Tensor], exp_avg: Sequence[torch.Tensor], exp_avg_sq: Sequence[torch.Tensor], *,
                  master: Optional[Sequence[torch.Tensor]] = None,
                  exp_avg_scales: Optional[Sequence[torch.Tensor]] = None,
                  exp_avg_sq_scales: Optional[Sequence[torch.Tensor]] = None) -> AdamwTensors:
    """Checks the tensors of an AdamW optimiser and returns their table for ``adamw_step``.

    params bfloat16 or float32 (all of one type), contiguous, any shapes; ``master`` the float32 weights behind them.
    exp_avg, exp_avg_sq: float32 of the params' sizes, or int8 and uint8 with a float32 scale for each 256 elements
    (exp_avg_scales, exp_avg_sq_scales).  Zeros are the state to start from.  The table names the tensors' memory: make it
    anew when that is replaced (``p.data = ...``).
    """
    if not params:
        raise ValueError("params must hold a tensor")
    dtype, dev = params[0].dtype, _gpu(params[0], "params")
    code = _dtype_code(params[0])
    bits = 8 if exp_avg and exp_avg[0].dtype == torch.int8 else 32
    types = (torch.int8, torch.uint8) if bits == 8 else (torch.float32, torch.float32)
    if (exp_avg_scales is None) != (bits == 32) or (exp_avg_sq_scales is None) != (bits == 32):
        raise ValueError("exp_avg_scales and exp_avg_sq_scales must be given exactly with 8-bit states")
    lists = [("params", "param", params, dtype), ("exp_avg", "exp_avg", exp_avg, types[0]),
             ("exp_avg_sq", "exp_avg_sq", exp_avg_sq, types[1]), ("master", "master", master, torch.float32),
             ("exp_avg_scales", "exp_avg_scale", exp_avg_scales, torch.float32),
             ("exp_avg_sq_scales", "exp_avg_sq_scale", exp_avg_sq_scales, torch.float32)]
    table = (_AdamwTensor * len(params))()
    sizes = [p.numel() for p in params]
    for name, field, tensors, dt in lists:
        if tensors is None:
            continue
        if len(tensors) != len(params):
            raise ValueError(f"{name} must hold {len(params)} tensors")
        for i, t in enumerate(tensors):
            need = -(-sizes[i] // 256) if name.endswith("scales") else sizes[i]
            if t.dtype != dt or t.numel() != need or not t.is_contiguous() or t.get_device() != dev:
                raise ValueError(f"{name}[{i}] must be a contiguous {dt} tensor of {need} elements on cuda:{dev}")
            setattr(table[i], field, t.data_ptr())
    for i, n in enumerate(sizes):
        table[i].n = n
    _check(load().ttt_adamw_check(table, len(params), bits, code))
    return AdamwTensors(table, sizes, dtype, bits, dev, [x[2] for x in lists if x[2] is not None],
                        [*params, *(master or ())])


def adamw_step(tensors: AdamwTensors, grads: Sequence[torch.Tensor], *, step, lr, betas: Tuple[float, float] = (0.9, 0.999),
               eps: float = 1e-8, weight_decay: float = 0.0, grad_scale: Optional[torch.Tensor] = None) -> None:
    """One AdamW step, in place on the params, masters and states of ``tensors``.

    grads: like the params.  step counts from 1; step (int64) and lr (float32) may be one-element GPU tensors, read when
    the kernels run (captured steps).  grad_scale: one-element float32 GPU tensor that multiplies every gradient.
    """
    dev, dtype, sizes, table = tensors.dev, tensors.dtype, tensors.sizes, tensors.table
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"the tensors must be on the current GPU, got cuda:{dev}")
    if len(grads) != len(sizes):
        raise ValueError(f"grads must hold {len(sizes)} tensors")
    if [t.data_ptr() for t in tensors.weights] != tensors.at:
        raise ValueError("params or masters have moved to other memory since adamw_tensors")
    for i, g in enumerate(grads):
        if g.dtype != dtype or g.numel() != sizes[i] or not g.is_contiguous() or g.get_device() != dev:
            raise ValueError(f"grads[{i}] must be a contiguous {dtype} tensor of {sizes[i]} elements on cuda:{dev}")
        table[i].grad = g.data_ptr()

    def scalar(t, dt, name):
        if t.dtype != dt or t.numel() != 1 or t.get_device() != dev:
            raise ValueError(f"{name} must be a one-element {dt} tensor on cuda:{dev}")
        return t.data_ptr()

    step_ptr = lr_ptr = workspace = None
    if isinstance(step, torch.Tensor):
        step_ptr, step = scalar(step, torch.int64, "step"), 1
    if isinstance(lr, torch.Tensor):
        lr_ptr, lr = scalar(lr, torch.float32, "lr"), 0.0
    if step_ptr is not None or lr_ptr is not None:
        workspace = torch.empty(16, dtype=torch.uint8, device=torch.device("cuda", dev))
    _check(load().ttt_adamw_step(table, len(sizes), int(step), step_ptr, float(lr), lr_ptr, float(betas[0]),
                                 float(betas[1]), float(eps), float(weight_decay),
                                 None if grad_scale is None else scalar(grad_scale, torch.float32, "grad_scale"),
                                 tensors.bits, TTT_BF16 if dtype == torch.bfloat16 else TTT_F32, _ptr(workspace),
                                 0 if workspace is None else 16, _stream()))


# ------------------------------------------------------------------ timing
def profile_enable(on: bool = True) -> None:
    _check(load().ttt_profile_enable(1 if on else 0))


def profile_reset() -> None:
    _check(load().ttt_profile_reset())


def profile_read() -> dict:
    """{kind: (total_ms, launches)} since the last reset (synchronises the timing events)."""
    res = {}
    for i, name in enumerate(KERNEL_KINDS):
        ms, cnt = ctypes.c_double(), ctypes.c_int64()
        _check(load().ttt_profile_read(i, ctypes.byref(ms), ctypes.byref(cnt)))
        res[name] = (ms.value, cnt.value)
    return res


def mfma_rate_probe(iters: int = 16384) -> float:
    """Launch the dense bf16 MFMA rate probe on the current stream; returns its FLOP count.

    Time the launch with events on the current stream to get the sustained rate."""
    flop = ctypes.c_double()
    _check(load().ttt_mfma_rate_probe(int(iters), _stream(), ctypes.byref(flop)))
    return flop.value
