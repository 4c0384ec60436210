"""Python binding of libtp_block.so (include/tp_block.h): argument marshalling only.

Every function here takes torch tensors that already live on the current CUDA
device, checks dtype / device / contiguity, and passes raw pointers, sizes and
the current stream to the C ABI of the same name.  All arithmetic runs in the
library's CUDA kernels; there is no fallback of any kind: if the shared library
is missing or fails to load, the first call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

from .build_lib import LIB_PATH

TP_OK = 0
TP_ERR_NULL = 1
TP_ERR_ALIGN = 2
TP_ERR_SHAPE = 3
TP_ERR_TP_DEGREE = 4
TP_ERR_WORKSPACE = 5
TP_ERR_UNSUPPORTED = 6
TP_ERR_CUDA = 7
TP_ERR_DEVICE_TIMEOUT = 8

TP_ACT_NONE = 0
TP_ACT_GELU_TANH = 1

TP_ROPE_HALF = 0
TP_ROPE_PAIRS = 1

TP_OPT_PDL = 1
TP_OPT_STATIC_WEIGHTS = 2

ACTS = {"none": TP_ACT_NONE, "gelu_tanh": TP_ACT_GELU_TANH}
ROPE_LAYOUTS = {"half": TP_ROPE_HALF, "pairs": TP_ROPE_PAIRS}

# name -> (restype, argtypes) of every symbol declared in include/tp_block.h
_P = ctypes.c_void_p
_I = ctypes.c_int
_Z = ctypes.c_size_t
_F = ctypes.c_float
SIGNATURES = {
    "tp_colpar_gemm_gelu": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P, _P]),
    "tp_rowpar_gemm_reduce": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "tp_mlp_workspace_bytes": (_Z, [_I, _I]),
    "tp_mlp_forward": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _Z, _P]),
    "tp_attn_proj_forward": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P]),
    "tp_mlp_forward_noalloc": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P]),
    "tp_mlp_backward_workspace_bytes": (_Z, [_I, _I]),
    "tp_attn_decode_workspace_bytes": (_Z, [_I, _I, _I, _I, _I]),
    "tp_sp_add_rmsnorm": (_I, [_P, _P, _P, _I, _I, _I, ctypes.c_float, _P, _P, _P]),
    "tp_attn_decode": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _Z, _P]),
    "tp_attn_prefill": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P]),
    "tp_qk_norm_rope": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P, _P]),
    "tp_qk_norm_rope_backward_workspace_bytes": (_Z, [_I, _I]),
    "tp_qk_norm_rope_backward": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I,
                                      _P, _P, _P, _P, _Z, _P]),
    "tp_kv_append": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P]),
    "tp_kv8_append": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P]),
    "tp_kv8_read": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _I, _P]),
    "tp_tree_mask": (_I, [_P, _I, _P]),
    "tp_attn_tree_workspace_bytes": (_Z, [_I, _I, _I, _I, _I]),
    "tp_attn_decode_kv8_workspace_bytes": (_Z, [_I, _I, _I, _I, _I]),
    "tp_attn_tree_workspace_bytes_upto": (_Z, [_I, _I, _I, _I, _I]),
    "tp_attn_tree": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _Z, _P]),
    "tp_attn_decode_kv8": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _Z,
                                _P]),
    "tp_mlp_backward": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _Z,
                             _P]),
    "tp_colpar_gemm_gelu_w8": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P]),
    "tp_rowpar_gemm_reduce_w8": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "tp_mlp_forward_w8": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _Z, _P]),
    "tp_status_string": (ctypes.c_char_p, [_I]),
    "tp_last_cuda_error": (ctypes.c_char_p, []),
    "tp_device_error_check": (_I, []),
    "tp_diag_bounded_wait": (_I, [ctypes.c_uint, _P, _P]),
    "tp_set_decode_max_tokens": (_I, [_I]),
    "tp_get_decode_max_tokens": (_I, []),
    "tp_set_launch_options": (_I, [ctypes.c_uint]),
    "tp_get_launch_options": (ctypes.c_uint, []),
    "tp_stream_plan": (_I, [_I, _I, _I, _I, _I, _I, _I, _P]),
}


class StreamPlan(ctypes.Structure):
    """tp_stream_plan_t of include/tp_block.h."""
    _fields_ = [(name, ctypes.c_int) for name in (
        "grid_x", "cluster", "jsplit", "shards_per_cta", "stages", "kblocks_per_box",
        "stage_bytes", "smem_bytes", "l2_ahead")]


# a B200: 148 multiprocessors, 227 KB of opt-in shared memory per block
B200_SMS = 148
B200_MAX_SMEM = 232448


class TPError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: status {status} ({status_string(status)})"
        if status == TP_ERR_CUDA:
            msg += f": {load().tp_last_cuda_error().decode()}"
        super().__init__(msg)


_lib: Optional[ctypes.CDLL] = None


def library_path() -> str:
    return LIB_PATH


def load() -> ctypes.CDLL:
    """Load the shared library (raises if it is absent: build it first)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing; build it with "
                "`python -m tensor_transformer_linear_column_b200.build_lib`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().tp_status_string(int(status)).decode()


def _ptr(t: Optional[torch.Tensor], name: str, dev: torch.device) -> Optional[int]:
    return _ptr_typed(t, name, dev, torch.bfloat16)


def _ptr_typed(t: Optional[torch.Tensor], name: str, dev: torch.device,
               dtype: torch.dtype) -> Optional[int]:
    """The pointer of a contiguous tensor of the given type on the call's device."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is dtype and t.device == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {str(dtype).replace('torch.', '')}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    raise ValueError(f"{name} must be contiguous")


def _device(t: torch.Tensor) -> torch.device:
    """The device of a call: that of its first tensor, which must be the current
    CUDA device (the library launches there; a host or other-device pointer
    handed to a kernel would fault)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("inputs must be CUDA tensors")
    dev = t.device
    cur = torch._C._cuda_getDevice()  # there is a CUDA tensor: nothing to initialise
    if dev.index != cur:
        raise ValueError(f"inputs are on {dev} but the current device is cuda:{cur}; "
                         f"call under torch.cuda.device({dev.index})")
    return dev


def _stream(stream: Optional[torch.cuda.Stream]) -> int:
    if stream is None:
        # the handle itself: a torch.cuda.Stream object costs 3 us to build
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if stream.device.index != torch.cuda.current_device():
        raise ValueError(f"stream is on {stream.device}, not the current device")
    return stream.cuda_stream


def _check(status: int, where: str) -> None:
    if status != TP_OK:
        raise TPError(status, where)


def _act(act) -> int:
    return ACTS[act] if isinstance(act, str) else int(act)


def tp_colpar_gemm_gelu(x: torch.Tensor, w: torch.Tensor, b: Optional[torch.Tensor],
                        tp_degree: int, act="none", out: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """out[T, N] = act(x[T, K] @ w[N, K]^T + b) with the output split in tp_degree shards."""
    T, K = x.shape
    N = w.shape[0]
    if w.shape[1] != K:
        raise ValueError("w must be [N, K]")
    dev = _device(x)
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
    st = load().tp_colpar_gemm_gelu(_ptr(x, "x", dev), _ptr(w, "w", dev), _ptr(b, "b", dev),
                                    T, K, N, int(tp_degree), _act(act), _ptr(out, "out", dev),
                                    _stream(stream))
    _check(st, "tp_colpar_gemm_gelu")
    return out


def tp_rowpar_gemm_reduce(h: torch.Tensor, w: torch.Tensor, b: Optional[torch.Tensor],
                          tp_degree: int, out: Optional[torch.Tensor] = None,
                          stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """out[T, N] = sum_s h[:, K_s] @ w[:, K_s]^T + b over tp_degree shards of K."""
    T, K = h.shape
    N = w.shape[0]
    if w.shape[1] != K:
        raise ValueError("w must be [N, K]")
    dev = _device(h)
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
    st = load().tp_rowpar_gemm_reduce(_ptr(h, "h", dev), _ptr(w, "w", dev), _ptr(b, "b", dev),
                                      T, K, N, int(tp_degree), _ptr(out, "out", dev),
                                      _stream(stream))
    _check(st, "tp_rowpar_gemm_reduce")
    return out


def tp_mlp_workspace_bytes(T: int, F: int) -> int:
    return int(load().tp_mlp_workspace_bytes(int(T), int(F)))


def tp_mlp_forward(x: torch.Tensor, w1: torch.Tensor, b1: Optional[torch.Tensor],
                   w2: torch.Tensor, b2: Optional[torch.Tensor], tp_degree: int,
                   act="gelu_tanh", out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The tensor-parallel MLP block y = sum_s act(x W1_s^T + b1_s) W2[:, s]^T + b2."""
    T, H = x.shape
    F = w1.shape[0]
    if w1.shape[1] != H or tuple(w2.shape) != (H, F):
        raise ValueError("w1 must be [F, H] and w2 [H, F]")
    dev = _device(x)
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    need = tp_mlp_workspace_bytes(T, F)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the same device")
    ws_bytes = workspace.numel() * workspace.element_size()
    st = load().tp_mlp_forward(_ptr(x, "x", dev), _ptr(w1, "w1", dev), _ptr(b1, "b1", dev),
                               _ptr(w2, "w2", dev), _ptr(b2, "b2", dev), T, H, F,
                               int(tp_degree), _act(act), _ptr(out, "out", dev),
                               workspace.data_ptr(), ws_bytes, _stream(stream))
    _check(st, "tp_mlp_forward")
    return out


def tp_mlp_backward_workspace_bytes(T: int, F: int) -> int:
    return int(load().tp_mlp_backward_workspace_bytes(int(T), int(F)))


def tp_mlp_backward(x: torch.Tensor, w1: torch.Tensor, b1: Optional[torch.Tensor],
                    w2: torch.Tensor, dy: torch.Tensor, tp_degree: int, act="gelu_tanh",
                    with_bias_grads: bool = True, workspace: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Gradients of the tensor-parallel MLP block for the upstream gradient dy:
    {"dx", "dw1", "db1", "dw2", "db2"} (the bias gradients only if asked)."""
    T, H = x.shape
    F = w1.shape[0]
    if w1.shape[1] != H or tuple(w2.shape) != (H, F) or tuple(dy.shape) != (T, H):
        raise ValueError("w1 must be [F, H], w2 [H, F] and dy [T, H]")
    dev = _device(x)
    out = {"dx": torch.empty((T, H), dtype=torch.bfloat16, device=dev),
           "dw1": torch.empty((F, H), dtype=torch.bfloat16, device=dev),
           "dw2": torch.empty((H, F), dtype=torch.bfloat16, device=dev),
           "db1": torch.empty((F,), dtype=torch.bfloat16, device=dev) if with_bias_grads else None,
           "db2": torch.empty((H,), dtype=torch.bfloat16, device=dev) if with_bias_grads else None}
    need = tp_mlp_backward_workspace_bytes(T, F)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the same device")
    st = load().tp_mlp_backward(
        _ptr(x, "x", dev), _ptr(w1, "w1", dev), _ptr(b1, "b1", dev), _ptr(w2, "w2", dev),
        _ptr(dy, "dy", dev), T, H, F, int(tp_degree), _act(act), _ptr(out["dx"], "dx", dev),
        _ptr(out["dw1"], "dw1", dev), _ptr(out["db1"], "db1", dev), _ptr(out["dw2"], "dw2", dev),
        _ptr(out["db2"], "db2", dev), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "tp_mlp_backward")
    return out


def tp_colpar_gemm_gelu_w8(x: torch.Tensor, w8: torch.Tensor, w_scale: torch.Tensor,
                           b: Optional[torch.Tensor], tp_degree: int, act="none",
                           out: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """tp_colpar_gemm_gelu with an 8-bit weight: w8 [N, K] E4M3 bytes (uint8) and
    w_scale [N] fp32, W[n, k] = w_scale[n] * e4m3(w8[n, k])."""
    T, K = x.shape
    N = w8.shape[0]
    if w8.shape[1] != K or tuple(w_scale.shape) != (N,):
        raise ValueError("w8 must be [N, K] and w_scale [N]")
    dev = _device(x)
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
    st = load().tp_colpar_gemm_gelu_w8(
        _ptr(x, "x", dev), _ptr_typed(w8, "w8", dev, torch.uint8),
        _ptr_typed(w_scale, "w_scale", dev, torch.float32), _ptr(b, "b", dev), T, K, N,
        int(tp_degree), _act(act), _ptr(out, "out", dev), _stream(stream))
    _check(st, "tp_colpar_gemm_gelu_w8")
    return out


def tp_rowpar_gemm_reduce_w8(h: torch.Tensor, w8: torch.Tensor, w_scale: torch.Tensor,
                             b: Optional[torch.Tensor], tp_degree: int,
                             out: Optional[torch.Tensor] = None,
                             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """tp_rowpar_gemm_reduce with an 8-bit weight (see tp_colpar_gemm_gelu_w8)."""
    T, K = h.shape
    N = w8.shape[0]
    if w8.shape[1] != K or tuple(w_scale.shape) != (N,):
        raise ValueError("w8 must be [N, K] and w_scale [N]")
    dev = _device(h)
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
    st = load().tp_rowpar_gemm_reduce_w8(
        _ptr(h, "h", dev), _ptr_typed(w8, "w8", dev, torch.uint8),
        _ptr_typed(w_scale, "w_scale", dev, torch.float32), _ptr(b, "b", dev), T, K, N,
        int(tp_degree), _ptr(out, "out", dev), _stream(stream))
    _check(st, "tp_rowpar_gemm_reduce_w8")
    return out


def tp_mlp_forward_w8(x: torch.Tensor, w1: torch.Tensor, s1: torch.Tensor,
                      b1: Optional[torch.Tensor], w2: torch.Tensor, s2: torch.Tensor,
                      b2: Optional[torch.Tensor], tp_degree: int, act="gelu_tanh",
                      out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """tp_mlp_forward with 8-bit weights: w1 [F, H] and w2 [H, F] E4M3 bytes,
    s1 [F] and s2 [H] fp32 row scales."""
    T, H = x.shape
    F = w1.shape[0]
    if w1.shape[1] != H or tuple(w2.shape) != (H, F):
        raise ValueError("w1 must be [F, H] and w2 [H, F]")
    if tuple(s1.shape) != (F,) or tuple(s2.shape) != (H,):
        raise ValueError("s1 must be [F] and s2 [H]")
    dev = _device(x)
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    need = tp_mlp_workspace_bytes(T, F)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the same device")
    ws_bytes = workspace.numel() * workspace.element_size()
    st = load().tp_mlp_forward_w8(
        _ptr(x, "x", dev), _ptr_typed(w1, "w1", dev, torch.uint8),
        _ptr_typed(s1, "s1", dev, torch.float32), _ptr(b1, "b1", dev),
        _ptr_typed(w2, "w2", dev, torch.uint8), _ptr_typed(s2, "s2", dev, torch.float32),
        _ptr(b2, "b2", dev), T, H, F, int(tp_degree), _act(act), _ptr(out, "out", dev),
        workspace.data_ptr(), ws_bytes, _stream(stream))
    _check(st, "tp_mlp_forward_w8")
    return out


TP_NOALLOC_SCRATCH_BYTES = 4 * 1024 * 1024


def tp_mlp_forward_noalloc(x: torch.Tensor, w1: torch.Tensor, b1: Optional[torch.Tensor],
                           w2: torch.Tensor, b2: Optional[torch.Tensor], tp_degree: int,
                           act="gelu_tanh", out: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """tp_mlp_forward without a workspace, for callers that cannot allocate device
    memory: h lives in the library's own TP_NOALLOC_SCRATCH_BYTES device array,
    shared by every call on the device (calls that may overlap on the GPU race)."""
    T, H = x.shape
    F = w1.shape[0]
    if w1.shape[1] != H or tuple(w2.shape) != (H, F):
        raise ValueError("w1 must be [F, H] and w2 [H, F]")
    dev = _device(x)
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    st = load().tp_mlp_forward_noalloc(_ptr(x, "x", dev), _ptr(w1, "w1", dev),
                                       _ptr(b1, "b1", dev), _ptr(w2, "w2", dev),
                                       _ptr(b2, "b2", dev), T, H, F, int(tp_degree), _act(act),
                                       _ptr(out, "out", dev), _stream(stream))
    _check(st, "tp_mlp_forward_noalloc")
    return out


def tp_attn_proj_forward(x: torch.Tensor, w_qkv: torch.Tensor, b_qkv: Optional[torch.Tensor],
                         ctx: torch.Tensor, w_o: torch.Tensor, b_o: Optional[torch.Tensor],
                         n_q_heads: int, n_kv_heads: int, head_dim: int, tp_degree: int,
                         qkv_out: Optional[torch.Tensor] = None,
                         out: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None):
    """(qkv, y): the head-split QKV projection and the row-parallel output projection."""
    T, H = x.shape
    dev = _device(x)
    nqkv = (n_q_heads + 2 * n_kv_heads) * head_dim
    if qkv_out is None:
        qkv_out = torch.empty((T, nqkv), dtype=torch.bfloat16, device=dev)
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    st = load().tp_attn_proj_forward(_ptr(x, "x", dev), _ptr(w_qkv, "w_qkv", dev),
                                     _ptr(b_qkv, "b_qkv", dev), _ptr(ctx, "ctx", dev),
                                     _ptr(w_o, "w_o", dev), _ptr(b_o, "b_o", dev), T, H,
                                     int(n_q_heads), int(n_kv_heads), int(head_dim),
                                     int(tp_degree), _ptr(qkv_out, "qkv_out", dev),
                                     _ptr(out, "out", dev), _stream(stream))
    _check(st, "tp_attn_proj_forward")
    return qkv_out, out


def tp_attn_decode_workspace_bytes(T: int, past: int, n_q_heads: int, n_kv_heads: int,
                                   head_dim: int) -> int:
    return int(load().tp_attn_decode_workspace_bytes(int(T), int(past), int(n_q_heads),
                                                     int(n_kv_heads), int(head_dim)))


def tp_attn_decode(qkv: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, past: int,
                   n_q_heads: int, n_kv_heads: int, head_dim: int, tp_degree: int,
                   ctx: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """ctx [T, nq d] of T new tokens (qkv [T, (nq + 2 nkv) d]) over the caches
    k_cache, v_cache [nkv, max_len, d] holding `past` tokens; appends the new
    tokens' keys and values to the caches in place."""
    T = qkv.shape[0]
    if qkv.shape[1] != (n_q_heads + 2 * n_kv_heads) * head_dim:
        raise ValueError("qkv must be [T, (nq + 2 nkv) d]")
    if k_cache.dim() != 3 or tuple(k_cache.shape) != tuple(v_cache.shape) or \
            k_cache.shape[0] != n_kv_heads or k_cache.shape[2] != head_dim:
        raise ValueError("caches must be [nkv, max_len, d]")
    dev = _device(qkv)
    if ctx is None:
        ctx = torch.empty((T, n_q_heads * head_dim), dtype=torch.bfloat16, device=dev)
    need = tp_attn_decode_workspace_bytes(T, past, n_q_heads, n_kv_heads, head_dim)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the same device")
    st = load().tp_attn_decode(_ptr(qkv, "qkv", dev), _ptr(k_cache, "k_cache", dev),
                               _ptr(v_cache, "v_cache", dev), T, int(past), k_cache.shape[1],
                               int(n_q_heads), int(n_kv_heads), int(head_dim), int(tp_degree),
                               _ptr(ctx, "ctx", dev), workspace.data_ptr(),
                               workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "tp_attn_decode")
    return ctx


def tp_attn_prefill(qkv: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, past: int,
                    n_q_heads: int, n_kv_heads: int, head_dim: int, tp_degree: int,
                    ctx: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The attention core for many new tokens at once (a prompt or a chunk of
    one): ctx [T, nq d] of qkv [T, (nq + 2 nkv) d] over the caches k_cache,
    v_cache [nkv, max_len, d] holding `past` tokens; appends the new tokens'
    keys and values to the caches in place.  Needs no workspace."""
    T = qkv.shape[0]
    if qkv.shape[1] != (n_q_heads + 2 * n_kv_heads) * head_dim:
        raise ValueError("qkv must be [T, (nq + 2 nkv) d]")
    if k_cache.dim() != 3 or tuple(k_cache.shape) != tuple(v_cache.shape) or \
            k_cache.shape[0] != n_kv_heads or k_cache.shape[2] != head_dim:
        raise ValueError("caches must be [nkv, max_len, d]")
    dev = _device(qkv)
    if ctx is None:
        ctx = torch.empty((T, n_q_heads * head_dim), dtype=torch.bfloat16, device=dev)
    st = load().tp_attn_prefill(_ptr(qkv, "qkv", dev), _ptr(k_cache, "k_cache", dev),
                                _ptr(v_cache, "v_cache", dev), T, int(past), k_cache.shape[1],
                                int(n_q_heads), int(n_kv_heads), int(head_dim), int(tp_degree),
                                _ptr(ctx, "ctx", dev), _stream(stream))
    _check(st, "tp_attn_prefill")
    return ctx


def tp_sp_add_rmsnorm(y: torch.Tensor, residual: torch.Tensor, gamma: torch.Tensor,
                      tp_degree: int, eps: float = 1e-5, r_out: Optional[torch.Tensor] = None,
                      n_out: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None):
    """(r, n): r = residual + y, n = RMSNorm(r) * gamma, by token shards of T / t."""
    T, H = y.shape
    if tuple(residual.shape) != (T, H) or tuple(gamma.shape) != (H,):
        raise ValueError("residual must be [T, H] and gamma [H]")
    dev = _device(y)
    if r_out is None:
        r_out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    if n_out is None:
        n_out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    st = load().tp_sp_add_rmsnorm(_ptr(y, "y", dev), _ptr(residual, "residual", dev),
                                  _ptr(gamma, "gamma", dev), T, H, int(tp_degree), float(eps),
                                  _ptr(r_out, "r_out", dev), _ptr(n_out, "n_out", dev),
                                  _stream(stream))
    _check(st, "tp_sp_add_rmsnorm")
    return r_out, n_out


def _empty_on(like: torch.Tensor, shape, stream: Optional[torch.cuda.Stream],
              dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """An uninitialised tensor on like's device (and of its type) whose memory
    belongs to the call's stream: it is handed out again only after the work
    enqueued there."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _workspace(workspace: Optional[torch.Tensor], need: int, like: torch.Tensor,
               dev: torch.device, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """The caller's workspace, or one of `need` bytes (like is bf16)."""
    if workspace is None:
        size = (max(need, 256) + 1) // 2
        return like.new_empty(size) if stream is None else _empty_on(like, size, stream)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the same device")
    return workspace


def _int32(value, name: str) -> int:
    """A length or position as the C int it is passed as (ctypes would wrap it)."""
    value = int(value)
    if not -2 ** 31 <= value < 2 ** 31:
        raise ValueError(f"{name} must fit 32 bits, got {value}")
    return value


def _expect_shape(t: Optional[torch.Tensor], name: str, shape) -> None:
    if t is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _qk_args(qkv, gamma_q, gamma_k, inv_freq, positions, n_q_heads, n_kv_heads, head_dim, dev):
    """Shape checks shared by tp_qk_norm_rope and its gradient; the pointers of
    the gains, the frequencies and the positions, and rot_dim."""
    shape = qkv.shape
    if len(shape) != 2 or shape[1] != (n_q_heads + 2 * n_kv_heads) * head_dim:
        raise ValueError("qkv must be [T, (nq + 2 nkv) d]")
    gq = gk = fr = pos = None
    rot = 0
    if gamma_q is not None or gamma_k is not None:
        _expect_shape(gamma_q, "gamma_q", (head_dim,))
        _expect_shape(gamma_k, "gamma_k", (head_dim,))
        gq = _ptr_typed(gamma_q, "gamma_q", dev, torch.bfloat16)
        gk = _ptr_typed(gamma_k, "gamma_k", dev, torch.bfloat16)
    if positions is not None:
        _expect_shape(positions, "positions", (shape[0],))
        pos = _ptr_typed(positions, "positions", dev, torch.int32)
    if inv_freq is not None:
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must be [rot_dim / 2]")
        rot = 2 * inv_freq.shape[0]
        if rot:
            fr = _ptr_typed(inv_freq, "inv_freq", dev, torch.float32)
    return gq, gk, fr, pos, rot


def _layout(layout) -> int:
    return ROPE_LAYOUTS[layout] if isinstance(layout, str) else int(layout)


def tp_qk_norm_rope(qkv: torch.Tensor, past: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                    tp_degree: int, gamma_q: Optional[torch.Tensor] = None,
                    gamma_k: Optional[torch.Tensor] = None,
                    inv_freq: Optional[torch.Tensor] = None,
                    positions: Optional[torch.Tensor] = None, layout="half", eps: float = 1e-5,
                    out: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """RMS norm of every query and key head (gamma_q, gamma_k [d], or neither) and
    the rotation of its first 2 len(inv_freq) elements by position * inv_freq:
    qkv [T, (nq + 2 nkv) d] to a buffer of the same shape, which may be qkv
    itself (out=qkv).  Token i is at positions[i] (int32), or at past + i;
    layout "half" pairs (p, p + rot / 2), "pairs" (2 p, 2 p + 1)."""
    past = _int32(past, "past")
    dev = _device(qkv)
    gq, gk, fr, pos, rot = _qk_args(qkv, gamma_q, gamma_k, inv_freq, positions, n_q_heads,
                                    n_kv_heads, head_dim, dev)
    if out is None:
        out = torch.empty_like(qkv) if stream is None else _empty_on(qkv, qkv.shape, stream)
    else:
        _expect_shape(out, "out", qkv.shape)
    st = load().tp_qk_norm_rope(_ptr(qkv, "qkv", dev), gq, gk, fr, pos, qkv.shape[0], past,
                                int(n_q_heads), int(n_kv_heads), int(head_dim), rot,
                                _layout(layout), float(eps), int(tp_degree),
                                _ptr(out, "out", dev), _stream(stream))
    _check(st, "tp_qk_norm_rope")
    return out


def tp_qk_norm_rope_backward_workspace_bytes(T: int, head_dim: int) -> int:
    return int(load().tp_qk_norm_rope_backward_workspace_bytes(int(T), int(head_dim)))


def tp_qk_norm_rope_backward(qkv: torch.Tensor, dout: torch.Tensor, past: int, n_q_heads: int,
                             n_kv_heads: int, head_dim: int, tp_degree: int,
                             gamma_q: Optional[torch.Tensor] = None,
                             gamma_k: Optional[torch.Tensor] = None,
                             inv_freq: Optional[torch.Tensor] = None,
                             positions: Optional[torch.Tensor] = None, layout="half",
                             eps: float = 1e-5, dqkv: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None,
                             stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Gradients of tp_qk_norm_rope for the upstream gradient dout of its result:
    {"dqkv", "dgamma_q", "dgamma_k"} (the gains' None without norms).  qkv is the
    forward call's input, so a forward call that is to be differentiated must not
    run in place; dqkv may be dout itself."""
    past = _int32(past, "past")
    dev = _device(qkv)
    gq, gk, fr, pos, rot = _qk_args(qkv, gamma_q, gamma_k, inv_freq, positions, n_q_heads,
                                    n_kv_heads, head_dim, dev)
    _expect_shape(dout, "dout", qkv.shape)
    T = qkv.shape[0]
    if dqkv is None:
        dqkv = _empty_on(qkv, qkv.shape, stream)
    else:
        _expect_shape(dqkv, "dqkv", qkv.shape)
    dgq = dgk = ws = None
    if gq is not None:
        dgq = _empty_on(qkv, head_dim, stream)
        dgk = _empty_on(qkv, head_dim, stream)
        ws = _workspace(workspace, tp_qk_norm_rope_backward_workspace_bytes(T, head_dim), qkv, dev,
                        stream)
    st = load().tp_qk_norm_rope_backward(
        _ptr(qkv, "qkv", dev), gq, gk, fr, pos, _ptr(dout, "dout", dev), T, past,
        int(n_q_heads), int(n_kv_heads), int(head_dim), rot, _layout(layout), float(eps),
        int(tp_degree), _ptr(dqkv, "dqkv", dev), _ptr(dgq, "dgamma_q", dev),
        _ptr(dgk, "dgamma_k", dev), None if ws is None else ws.data_ptr(),
        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "tp_qk_norm_rope_backward")
    return {"dqkv": dqkv, "dgamma_q": dgq, "dgamma_k": dgk}


def _check_qkv_cache(qkv, k_cache, v_cache, n_q_heads, n_kv_heads, head_dim):
    """T and max_len."""
    rows, shape = qkv.shape, k_cache.shape
    if len(rows) != 2 or rows[1] != (n_q_heads + 2 * n_kv_heads) * head_dim:
        raise ValueError("qkv must be [T, (nq + 2 nkv) d]")
    if len(shape) != 3 or shape != v_cache.shape or shape[0] != n_kv_heads or \
            shape[2] != head_dim:
        raise ValueError("caches must be [nkv, max_len, d]")
    return rows[0], _int32(shape[1], "max_len")


def _kv8_ptrs(k_cache, k_scale, v_cache, v_scale, shape, dev):
    """The pointers of an 8-bit cache whose scales are [nkv, max_len] = shape."""
    _expect_shape(k_scale, "k_scale", shape)
    _expect_shape(v_scale, "v_scale", shape)
    return (_ptr_typed(k_cache, "k_cache", dev, torch.uint8),
            _ptr_typed(k_scale, "k_scale", dev, torch.float32),
            _ptr_typed(v_cache, "v_cache", dev, torch.uint8),
            _ptr_typed(v_scale, "v_scale", dev, torch.float32))


def _rows(rows, T, dev):
    """(pointer, count) of the rows to append; all T without a list."""
    if rows is None:
        return None, T
    if rows.dim() != 1:
        raise ValueError("rows must be [n]")
    return _ptr_typed(rows, "rows", dev, torch.int32), rows.shape[0]


def tp_kv_append(qkv: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, past: int,
                 n_q_heads: int, n_kv_heads: int, head_dim: int, tp_degree: int,
                 rows: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> None:
    """Write the keys and values of qkv's rows (int32 `rows` in that order, or all
    T) into the bf16 caches [nkv, max_len, d] from row `past` on, in place."""
    T, max_len = _check_qkv_cache(qkv, k_cache, v_cache, n_q_heads, n_kv_heads, head_dim)
    past = _int32(past, "past")
    dev = _device(qkv)
    rp, n = _rows(rows, T, dev)
    _check(load().tp_kv_append(_ptr(qkv, "qkv", dev), rp, _ptr(k_cache, "k_cache", dev),
                               _ptr(v_cache, "v_cache", dev), T, n, past,
                               max_len, int(n_q_heads), int(n_kv_heads), int(head_dim),
                               int(tp_degree), _stream(stream)), "tp_kv_append")


def tp_kv8_append(qkv: torch.Tensor, k_cache: torch.Tensor, k_scale: torch.Tensor,
                  v_cache: torch.Tensor, v_scale: torch.Tensor, past: int, n_q_heads: int,
                  n_kv_heads: int, head_dim: int, tp_degree: int,
                  rows: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> None:
    """tp_kv_append into an 8-bit cache: E4M3 codes (uint8) [nkv, max_len, d] and
    fp32 scales [nkv, max_len], a row being scale * e4m3(code)."""
    T, max_len = _check_qkv_cache(qkv, k_cache, v_cache, n_q_heads, n_kv_heads, head_dim)
    past = _int32(past, "past")
    dev = _device(qkv)
    rp, n = _rows(rows, T, dev)
    _check(load().tp_kv8_append(_ptr(qkv, "qkv", dev), rp,
                                *_kv8_ptrs(k_cache, k_scale, v_cache, v_scale,
                                           (n_kv_heads, max_len), dev), T,
                                n, past, max_len, int(n_q_heads), int(n_kv_heads),
                                int(head_dim), int(tp_degree), _stream(stream)), "tp_kv8_append")


def tp_kv8_read(k_cache: torch.Tensor, k_scale: torch.Tensor, v_cache: torch.Tensor,
                v_scale: torch.Tensor, start: int, count: int, tp_degree: int,
                k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None):
    """(k, v): rows [start, start + count) of an 8-bit cache as bf16 in the same
    rows of bf16 caches [nkv, out_len, d]; caches that are made here have
    out_len = start + count, their rows before `start` unset."""
    if k_cache.dim() != 3 or tuple(k_cache.shape) != tuple(v_cache.shape):
        raise ValueError("caches must be [nkv, max_len, d]")
    start, count = _int32(start, "start"), _int32(count, "count")
    nkv, max_len, d = k_cache.shape
    _int32(max_len, "max_len")
    dev = _device(k_cache)
    # (a range past max_len is refused below: no memory for it)
    shape = tuple((k_out if k_out is not None else v_out).shape) \
        if k_out is not None or v_out is not None \
        else (nkv, min(max(start + count, 1), max_len), d)
    if len(shape) != 3 or (shape[0], shape[2]) != (nkv, d):
        raise ValueError("k_out and v_out must be [nkv, out_len, d]")
    if k_out is None:
        k_out = _empty_on(k_cache, shape, stream, torch.bfloat16)
    if v_out is None:
        v_out = _empty_on(k_cache, shape, stream, torch.bfloat16)
    _expect_shape(v_out, "v_out", k_out.shape)
    _check(load().tp_kv8_read(*_kv8_ptrs(k_cache, k_scale, v_cache, v_scale, (nkv, max_len), dev),
                              start, count, max_len, nkv, d, int(tp_degree),
                              _ptr(k_out, "k_out", dev), _ptr(v_out, "v_out", dev),
                              _int32(shape[1], "out_len"), _stream(stream)), "tp_kv8_read")
    return k_out, v_out


def tp_tree_mask(parents) -> torch.Tensor:
    """Visibility words of a drafted tree, int64 [T, ceil(T / 64)] on the host:
    token i sees itself and its ancestors; parents[i] < i is the parent of token
    i, or -1 (host arithmetic, no GPU needed)."""
    parents = [_int32(v, "a parent") for v in parents]
    T = len(parents)
    words = torch.zeros((max(T, 1), max((T + 63) // 64, 1)), dtype=torch.int64)
    host = (ctypes.c_int32 * max(T, 1))(*parents)
    _check(load().tp_tree_mask(ctypes.addressof(host), T, words.data_ptr()), "tp_tree_mask")
    return words


def tp_attn_tree_workspace_bytes(T: int, past: int, n_q_heads: int, n_kv_heads: int,
                                 head_dim: int) -> int:
    return int(load().tp_attn_tree_workspace_bytes(_int32(T, "T"), _int32(past, "past"), int(n_q_heads),
                                                   int(n_kv_heads), int(head_dim)))


def tp_attn_decode_kv8_workspace_bytes(T: int, past: int, n_q_heads: int, n_kv_heads: int,
                                       head_dim: int) -> int:
    return int(load().tp_attn_decode_kv8_workspace_bytes(_int32(T, "T"), _int32(past, "past"), int(n_q_heads),
                                                         int(n_kv_heads), int(head_dim)))


def tp_attn_tree_workspace_bytes_upto(T: int, max_past: int, n_q_heads: int, n_kv_heads: int,
                                      head_dim: int) -> int:
    """Enough for tp_attn_tree and tp_attn_decode_kv8 after any number of cached
    tokens up to max_past; what the two above give may fall as `past` grows."""
    return int(load().tp_attn_tree_workspace_bytes_upto(_int32(T, "T"), _int32(max_past, "max_past"), int(n_q_heads),
                                                        int(n_kv_heads), int(head_dim)))


@functools.lru_cache(maxsize=256)
def _tree_workspace(name: str, T: int, blocks: int, n_q_heads: int, n_kv_heads: int,
                    head_dim: int) -> int:
    """The workspace of a call for `blocks` blocks of 128 cached tokens (the size
    depends on `past` through them alone)."""
    return getattr(load(), name + "_workspace_bytes")(T, 128 * blocks, n_q_heads, n_kv_heads,
                                                      head_dim)


def _tree_call(name, qkv, cache_ptrs, T, max_len, past, n_q_heads, n_kv_heads, head_dim, tp_degree,
               tree_mask, ctx, workspace, stream, dev) -> torch.Tensor:
    past, nq, nkv, d = _int32(past, "past"), int(n_q_heads), int(n_kv_heads), int(head_dim)
    mask = None
    if tree_mask is not None:
        _expect_shape(tree_mask, "tree_mask", (T, (T + 63) // 64))
        mask = _ptr_typed(tree_mask, "tree_mask", dev, torch.int64)
    if ctx is None:
        ctx = qkv.new_empty((T, nq * d)) if stream is None else _empty_on(qkv, (T, nq * d), stream)
    else:
        _expect_shape(ctx, "ctx", (T, nq * d))
    need = _tree_workspace(name, T, (past + 127) // 128, nq, nkv, d)
    ws_ptr, size = None, 0
    if workspace is not None or need > 0:
        ws = _workspace(workspace, need, qkv, dev, stream)
        ws_ptr, size = ws.data_ptr(), ws.numel() * ws.element_size()
    st = getattr(load(), name)(
        _ptr_typed(qkv, "qkv", dev, torch.bfloat16), *cache_ptrs, mask, T, past, max_len, nq, nkv,
        d, int(tp_degree), _ptr_typed(ctx, "ctx", dev, torch.bfloat16), ws_ptr, size,
        _stream(stream))
    _check(st, name)
    return ctx


def tp_attn_tree(qkv: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, past: int,
                 n_q_heads: int, n_kv_heads: int, head_dim: int, tp_degree: int,
                 tree_mask: Optional[torch.Tensor] = None, ctx: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """ctx [T, nq d] of T drafted tokens (T <= 128) over bf16 caches
    [nkv, max_len, d] that hold `past` tokens: every token sees those, and the
    new tokens that its row of tree_mask names (int64 words on the GPU, see
    tp_tree_mask; None: causal).  Writes the new tokens' keys and values behind
    the cached ones, in place."""
    T, max_len = _check_qkv_cache(qkv, k_cache, v_cache, n_q_heads, n_kv_heads, head_dim)
    dev = _device(qkv)
    return _tree_call("tp_attn_tree", qkv,
                      (_ptr(k_cache, "k_cache", dev), _ptr(v_cache, "v_cache", dev)),
                      T, max_len, past, n_q_heads, n_kv_heads, head_dim, tp_degree,
                      tree_mask, ctx, workspace, stream, dev)


def tp_attn_decode_kv8(qkv: torch.Tensor, k_cache: torch.Tensor, k_scale: torch.Tensor,
                       v_cache: torch.Tensor, v_scale: torch.Tensor, past: int, n_q_heads: int,
                       n_kv_heads: int, head_dim: int, tp_degree: int,
                       tree_mask: Optional[torch.Tensor] = None,
                       ctx: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """tp_attn_tree over an 8-bit cache (codes uint8 [nkv, max_len, d], scales
    fp32 [nkv, max_len]); decode when tree_mask is None.  The new tokens are
    quantised as they are written, and attended to as written."""
    T, max_len = _check_qkv_cache(qkv, k_cache, v_cache, n_q_heads, n_kv_heads, head_dim)
    dev = _device(qkv)
    return _tree_call("tp_attn_decode_kv8", qkv,
                      _kv8_ptrs(k_cache, k_scale, v_cache, v_scale, (n_kv_heads, max_len), dev),
                      T, max_len, past, n_q_heads, n_kv_heads, head_dim, tp_degree, tree_mask, ctx, workspace,
                      stream, dev)


def tp_device_error_check() -> int:
    """Synchronise, then read and clear the kernels' device-side error word."""
    return int(load().tp_device_error_check())


def tp_diag_bounded_wait(limit_us: int, result: torch.Tensor,
                         stream: Optional[torch.cuda.Stream] = None) -> None:
    """Diagnostic: a kernel whose bounded waits run out on purpose (result: int32[3]
    on the current device; see include/tp_block.h)."""
    dev = _device(result)
    if result.dtype != torch.int32 or result.numel() < 3 or not result.is_contiguous():
        raise ValueError("result must be a contiguous int32 tensor of at least 3 elements")
    if result.device != dev:
        raise ValueError("result must be on the current device")
    _check(load().tp_diag_bounded_wait(int(limit_us), result.data_ptr(), _stream(stream)),
           "tp_diag_bounded_wait")


def tp_set_decode_max_tokens(max_tokens: int) -> None:
    _check(load().tp_set_decode_max_tokens(int(max_tokens)), "tp_set_decode_max_tokens")


def tp_get_decode_max_tokens() -> int:
    return int(load().tp_get_decode_max_tokens())


def tp_stream_plan(T: int, K: int, N: int, row_shards: int = 1, w8: bool = False,
                   sms: int = B200_SMS, max_smem: int = B200_MAX_SMEM) -> dict:
    """The weight-streaming kernel's launch for one layer (host arithmetic, no GPU
    needed); raises TPError (e.g. TP_ERR_UNSUPPORTED) when it would not stream."""
    plan = StreamPlan()
    st = load().tp_stream_plan(int(T), int(K), int(N), int(row_shards), 1 if w8 else 0,
                               int(sms), int(max_smem), ctypes.addressof(plan))
    _check(st, "tp_stream_plan")
    return {name: getattr(plan, name) for name, _ in StreamPlan._fields_}


def tp_set_launch_options(flags: int) -> None:
    """TP_OPT_PDL | TP_OPT_STATIC_WEIGHTS (see include/tp_block.h)."""
    _check(load().tp_set_launch_options(int(flags)), "tp_set_launch_options")


def tp_get_launch_options() -> int:
    return int(load().tp_get_launch_options())
