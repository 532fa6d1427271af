"""Thin ctypes binding over libdiffattn.so (argument marshalling only).

Every computation runs in the library's CUDA kernels; this module checks
tensor placement/dtype/contiguity, passes raw device pointers, sizes and the
current CUDA stream, and turns a non-OK status into an exception.  PyTorch is
used only for device memory and streams.  If the library is missing this
module raises on first use: there is no fallback path.
"""

from __future__ import annotations

import ctypes
import functools
import operator
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# DIFFATTN_DEBUG=1 loads the bounds-check build (every TMA coordinate, TMEM
# address and global store of the kernels checked; see build.py) instead.
BOUNDS = os.environ.get("DIFFATTN_DEBUG", "") == "1"
LIB_PATH = os.path.join(_PKG, "libdiffattn_bounds.so" if BOUNDS else "libdiffattn.so")

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_DTYPE, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_BOUNDS = range(9)
STATUS_NAMES = ["OK", "ERR_NULL", "ERR_SHAPE", "ERR_ALIGN", "ERR_DTYPE", "ERR_UNSUPPORTED", "ERR_CUDA",
                "ERR_TIMEOUT", "ERR_BOUNDS"]
F32, BF16 = 0, 1

_lock = threading.Lock()
_lib = None


class DiffAttnError(RuntimeError):
    def __init__(self, status: int, msg: str):
        self.status = status
        name = STATUS_NAMES[status] if 0 <= status < len(STATUS_NAMES) else str(status)
        super().__init__(f"{name}: {msg}")


def lib() -> ctypes.CDLL:
    """Load libdiffattn.so (built in-tree by ``build.py``); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                   "`python -m differential_attention_03_gb300.build`"
                                   + (" --bounds" if BOUNDS else ""))
            L = ctypes.CDLL(LIB_PATH)
            vp, i, f, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong
            L.diffattn_lambda_init.argtypes = [i]
            L.diffattn_lambda_init.restype = f
            L.lambda_reparam.argtypes = [vp, vp, vp, vp, i, f, vp, vp]
            L.lambda_reparam.restype = i
            L.diffattn_forward.argtypes = [i, i, i, i, i, vp, vp, vp, vp, vp, vp, f, vp, f, i, vp, vp]
            L.diffattn_forward.restype = i
            L.diffattn_forward_host_workspace.argtypes = [i, i, i, i, i]
            L.diffattn_forward_host_workspace.restype = ctypes.c_size_t
            L.diffattn_forward_host.argtypes = [i, i, i, i, i, vp, vp, vp, vp, vp, vp, f, vp, f, i, vp, vp,
                                                ctypes.c_size_t, vp]
            L.diffattn_forward_host.restype = i
            L.diffattn_decode_workspace.argtypes = [i, i, i]
            L.diffattn_decode_workspace.restype = ctypes.c_size_t
            L.diffattn_v2_decode_workspace.argtypes = [i, i, i]
            L.diffattn_v2_decode_workspace.restype = ctypes.c_size_t
            L.diffattn_decode.argtypes = [i, i, i, i, i, vp, vp, vp, vp, vp, vp, vp, f, vp, f, vp, vp,
                                          ctypes.c_size_t, vp]
            L.diffattn_decode.restype = i
            L.diffattn_decode_noalloc.argtypes = [i, i, i, i, i, vp, vp, vp, vp, vp, vp, vp, f, vp, f, vp, vp]
            L.diffattn_decode_noalloc.restype = i
            L.diffattn_v2_decode.argtypes = [i, i, i, i, i, i, vp, vp, vp, vp, vp, ll, f, vp, vp, ctypes.c_size_t,
                                             vp]
            L.diffattn_v2_decode.restype = i
            L.diffattn_decode_fp8k.argtypes = [i, i, i, i, vp, vp, vp, vp, f, f, vp, vp, vp, f, vp, f, vp, vp,
                                               ctypes.c_size_t, vp]
            L.diffattn_decode_fp8k.restype = i
            L.diffattn_v2_decode_fp8k.argtypes = [i, i, i, i, i, vp, vp, f, vp, vp, vp, ll, f, vp, vp,
                                                  ctypes.c_size_t, vp]
            L.diffattn_v2_decode_fp8k.restype = i
            L.diffattn_backward_workspace.argtypes = [i, i, i, i]
            L.diffattn_backward_workspace.restype = ctypes.c_size_t
            L.diffattn_backward.argtypes = [i, i, i, i, i, vp, vp, vp, vp, vp, vp, f, vp, f, i, vp, vp, vp, vp, vp,
                                            vp, vp, vp, vp, ctypes.c_size_t, vp]
            L.diffattn_backward.restype = i
            L.diffattn_v2_backward_workspace.argtypes = [i, i, i, i]
            L.diffattn_v2_backward_workspace.restype = ctypes.c_size_t
            L.diffattn_v2_backward.argtypes = [i, i, i, i, i, i, vp, vp, vp, vp, ll, ll, f, i, vp, vp, vp, vp, vp,
                                               vp, ctypes.c_size_t, vp]
            L.diffattn_v2_backward.restype = i
            L.lambda_reparam_backward.argtypes = [vp, vp, vp, vp, i, vp, vp, vp, vp, vp, vp]
            L.lambda_reparam_backward.restype = i
            L.diffattn_v2_forward.argtypes = [i, i, i, i, i, i, vp, vp, vp, vp, ll, ll, f, i, vp, vp]
            L.diffattn_v2_forward.restype = i
            L.diffattn_forward_fp8qk.argtypes = [i, i, i, i, vp, vp, vp, vp, f, f, f, f, vp, vp, f, vp, f, i, vp, vp]
            L.diffattn_forward_fp8qk.restype = i
            L.diffattn_v2_forward_fp8qk.argtypes = [i, i, i, i, i, vp, vp, f, f, vp, vp, ll, ll, f, i, vp, vp]
            L.diffattn_v2_forward_fp8qk.restype = i
            sz = ctypes.c_size_t
            L.diffattn_forward_saved_bytes.argtypes = [i, i, i, i]
            L.diffattn_forward_saved_bytes.restype = sz
            L.diffattn_v2_forward_saved_bytes.argtypes = [i, i, i, i]
            L.diffattn_v2_forward_saved_bytes.restype = sz
            L.diffattn_forward_train.argtypes = [i, i, i, i, vp, vp, vp, vp, vp, vp, f, vp, f, i, vp, vp, sz, vp]
            L.diffattn_forward_train.restype = i
            L.diffattn_backward_saved.argtypes = [i, i, i, i, vp, vp, vp, vp, vp, vp, f, vp, f, i, vp, vp, sz,
                                                  vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
            L.diffattn_backward_saved.restype = i
            L.diffattn_v2_forward_train.argtypes = [i, i, i, i, i, vp, vp, vp, vp, ll, ll, f, i, vp, vp, sz, vp]
            L.diffattn_v2_forward_train.restype = i
            L.diffattn_v2_backward_saved.argtypes = [i, i, i, i, i, vp, vp, vp, vp, ll, ll, f, i, vp, vp, sz,
                                                     vp, vp, vp, vp, vp, sz, vp]
            L.diffattn_v2_backward_saved.restype = i
            L.diffattn_projection.argtypes = [i, i, i, vp, vp, vp, vp]
            L.diffattn_projection.restype = i
            L.diffattn_layer_workspace.argtypes = [i, i, i, i]
            L.diffattn_layer_workspace.restype = ctypes.c_size_t
            L.diffattn_layer_forward.argtypes = [i, i, i, i, i, vp, vp, vp, vp, vp, vp, vp, f, vp, f, i, vp, vp,
                                                 ctypes.c_size_t, vp]
            L.diffattn_layer_forward.restype = i
            L.diffattn_v2_layer_workspace.argtypes = [i, i, i, i, i]
            L.diffattn_v2_layer_workspace.restype = ctypes.c_size_t
            L.diffattn_v2_layer_forward.argtypes = [i, i, i, i, i, i, vp, vp, vp, i, vp, vp, ctypes.c_size_t, vp]
            L.diffattn_v2_layer_forward.restype = i
            d_ = ctypes.c_double
            L.diffattn_rope_init.argtypes = [vp, i, i, d_, i, d_, i, d_, d_]
            L.diffattn_rope_init.restype = i
            L.diffattn_rope_from_frequencies.argtypes = [vp, i, i, vp, f]
            L.diffattn_rope_from_frequencies.restype = i
            L.diffattn_rope.argtypes = [i, i, i, i, i, vp, vp, vp, vp, i, vp, vp]
            L.diffattn_rope.restype = i
            L.diffattn_cache_append.argtypes = [i, i, i, i, i, i] + [vp] * 14 + [f, f] + [vp] * 4
            L.diffattn_cache_append.restype = i
            L.diffattn_v2_cache_append.argtypes = [i, i, i, i, i, i, i] + [vp] * 10 + [f] + [vp] * 3
            L.diffattn_v2_cache_append.restype = i
            L.diffattn_cache_keep.argtypes = [i, i, i, i, i, i] + [vp] * 11
            L.diffattn_cache_keep.restype = i
            L.diffattn_v2_cache_keep.argtypes = [i, i, i, i, i, i] + [vp] * 9
            L.diffattn_v2_cache_keep.restype = i
            L.diffattn_tree_decode_workspace.argtypes = [i, i, i, i]
            L.diffattn_tree_decode_workspace.restype = sz
            L.diffattn_tree_decode.argtypes = [i, i, i, i, i, i, vp, vp, vp, vp, f, f, vp, vp, vp, vp, vp, vp, vp, ll,
                                               vp, f, vp, f, vp, vp, sz, vp]
            L.diffattn_tree_decode.restype = i
            L.diffattn_v2_tree_decode_workspace.argtypes = [i, i, i, i, i]
            L.diffattn_v2_tree_decode_workspace.restype = sz
            L.diffattn_v2_tree_decode.argtypes = [i, i, i, i, i, i, i, vp, vp, f, vp, vp, vp, vp, vp, vp, ll, vp, ll,
                                                  ll, f, vp, vp, sz, vp]
            L.diffattn_v2_tree_decode.restype = i
            L.diffattn_linear.argtypes = [i, i, i, vp, ll, vp, vp, i, vp, ll, i, vp, ll, vp, vp]
            L.diffattn_linear.restype = i
            L.diffattn_linear_backward_workspace.argtypes = [i, i, i]
            L.diffattn_linear_backward_workspace.restype = sz
            L.diffattn_linear_backward_workspace_for.argtypes = [i, i, i, i, i]
            L.diffattn_linear_backward_workspace_for.restype = sz
            L.diffattn_linear_backward.argtypes = [i, i, i, vp, ll, vp, vp, ll, vp, i, vp, vp, i, vp, vp, sz, vp]
            L.diffattn_linear_backward.restype = i
            L.diffattn_gated_linear.argtypes = [i, i, i, vp, ll, vp, i, vp, ll, vp, vp]
            L.diffattn_gated_linear.restype = i
            L.diffattn_gated_linear_backward_workspace.argtypes = [i, i, i]
            L.diffattn_gated_linear_backward_workspace.restype = sz
            L.diffattn_gated_linear_backward.argtypes = [i, i, i, vp, ll, vp, vp, vp, ll, i, vp, vp, i, vp, sz, vp]
            L.diffattn_gated_linear_backward.restype = i
            L.diffattn_residual_norm.argtypes = [i, i, i, i, vp, vp, vp, i, f, i, vp, vp, f, vp, vp, vp]
            L.diffattn_residual_norm.restype = i
            L.diffattn_residual_norm_backward_workspace.argtypes = [i, i, i]
            L.diffattn_residual_norm_backward_workspace.restype = sz
            L.diffattn_residual_norm_backward.argtypes = [i, i, i, i, vp, vp, vp, vp, vp, i, f, i, vp, vp, f] + [vp] * 6 + [sz, vp]
            L.diffattn_residual_norm_backward.restype = i
            L.diffattn_device_status.argtypes = [vp]
            L.diffattn_device_status.restype = i
            L.diffattn_bounds_checked.argtypes = []
            L.diffattn_bounds_checked.restype = i
            L.diffattn_debug_bounds_selftest.argtypes = [vp]
            L.diffattn_debug_bounds_selftest.restype = i
            L.diffattn_debug_item_plan.argtypes = [i, ll, i, i, i, i, ll, vp, vp]
            L.diffattn_debug_item_plan.restype = i
            L.diffattn_debug_product_plan.argtypes = [i, i, i, i, i, vp]
            L.diffattn_debug_product_plan.restype = i
            L.diffattn_last_error.argtypes = []
            L.diffattn_last_error.restype = ctypes.c_char_p
            L.diffattn_debug_wait_timeout.argtypes = [ll, vp]
            L.diffattn_debug_wait_timeout.restype = i
            L.diffattn_launch_count.argtypes = []
            L.diffattn_launch_count.restype = ll
            _lib = L
    return _lib


def _check(status: int):
    if status != OK:
        raise DiffAttnError(status, lib().diffattn_last_error().decode(errors="replace"))


def _stream(stream=None) -> int:
    if stream is None:  # (without the Stream object that torch.cuda.current_stream() makes: 3 us a call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t: torch.Tensor, name: str, dtype=None, shape=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise ValueError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def lambda_init(layer_index: int) -> float:
    """lambda_init = 0.8 - 0.6 exp(-0.3 (l - 1)) for the 1-based layer index (host)."""
    return float(lib().diffattn_lambda_init(int(layer_index)))


def lambda_reparam(lq1, lk1, lq2, lk2, lambda_init_value: float, out=None, stream=None) -> torch.Tensor:
    """Device scalar lambda = exp(lq1.lk1) - exp(lq2.lk2) + lambda_init (fp32, one element)."""
    for name, t in (("lq1", lq1), ("lk1", lk1), ("lq2", lq2), ("lk2", lk2)):
        _need(t, name, torch.float32, (lq1.numel(),))
    if out is None:
        out = torch.empty(1, device=lq1.device, dtype=torch.float32)
    _need(out, "out", torch.float32, (1,))
    _check(lib().lambda_reparam(_ptr(lq1), _ptr(lk1), _ptr(lq2), _ptr(lk2), lq1.numel(),
                                float(lambda_init_value), _ptr(out), _stream(stream)))
    return out


def diffattn_forward(q1, q2, k1, k2, v, lam, lambda_init_value: float, gamma=None, eps: float = 1e-5,
                     causal: bool = True, out=None, stream=None) -> torch.Tensor:
    """DIFF V1 forward with per-head RMSNorm x (1 - lambda_init); BSHD tensors.

    q1, q2, k1, k2: [B, n, H, d]; v: [B, n, H, 2d]; lam: device fp32 scalar
    tensor; gamma: fp32 [2d] or None.  Returns out [B, n, H, 2d] (input dtype).
    """
    B, n, H, d = q1.shape
    dt = q1.dtype
    for name, t in (("q1", q1), ("q2", q2), ("k1", k1), ("k2", k2)):
        _need(t, name, dt, (B, n, H, d))
    _need(v, "v", dt, (B, n, H, 2 * d))
    _need(lam, "lambda", torch.float32, (1,))
    if gamma is not None:
        _need(gamma, "gamma", torch.float32, (2 * d,))
    if out is None:
        out = torch.empty((B, n, H, 2 * d), device=q1.device, dtype=dt)
    _need(out, "out", dt, (B, n, H, 2 * d))
    _check(lib().diffattn_forward(_dt(q1), B, H, n, d, _ptr(q1), _ptr(q2), _ptr(k1), _ptr(k2), _ptr(v),
                                  _ptr(lam), float(lambda_init_value), _ptr(gamma), float(eps),
                                  1 if causal else 0, _ptr(out), _stream(stream)))
    return out


def diffattn_forward_fp8qk(q1, q2, k1, k2, scales, v, lam, lambda_init_value: float, gamma=None, eps: float = 1e-5,
                           causal: bool = True, out=None, stream=None) -> torch.Tensor:
    """DIFF V1 forward with e4m3 queries and keys (QK^T on the FP8 tensor-core path).

    q1, q2, k1, k2: [B, n, H, d] e4m3 codes (torch.float8_e4m3fn or their bytes as uint8) of
    Q_r / q_scale_r and K_r / k_scale_r, d = 128, or d = 64 with H >= 2; scales = (q1_scale,
    q2_scale, k1_scale, k2_scale).  The result is diffattn_forward's for Q_r = q_scale_r e4m3(q_r),
    K_r = k_scale_r e4m3(k_r); v bf16 [B, n, H, 2d].  Returns out [B, n, H, 2d] bf16.
    """
    B, n, H, d = q1.shape
    for name, t in (("q1", q1), ("q2", q2), ("k1", k1), ("k2", k2)):
        _need_fp8(t, name, (B, n, H, d))
    _need(v, "v", torch.bfloat16, (B, n, H, 2 * d))
    _need(lam, "lambda", torch.float32, (1,))
    if gamma is not None:
        _need(gamma, "gamma", torch.float32, (2 * d,))
    if out is None:
        out = torch.empty((B, n, H, 2 * d), device=v.device, dtype=torch.bfloat16)
    _need(out, "out", torch.bfloat16, (B, n, H, 2 * d))
    s1, s2, s3, s4 = (float(x) for x in scales)
    _check(lib().diffattn_forward_fp8qk(B, H, n, d, _ptr(q1), _ptr(q2), _ptr(k1), _ptr(k2), s1, s2, s3, s4, _ptr(v),
                                        _ptr(lam), float(lambda_init_value), _ptr(gamma), float(eps),
                                        1 if causal else 0, _ptr(out), _stream(stream)))
    return out


def _need_host(t: torch.Tensor, name: str, dtype=None, shape=None):
    if t.is_cuda:
        raise ValueError(f"{name} must be a host (CPU) tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def forward_host_workspace_bytes(dtype, B: int, H: int, n: int, d: int) -> int:
    """Device workspace (bytes) that diffattn_forward_host needs for these sizes."""
    return int(lib().diffattn_forward_host_workspace(BF16 if dtype == torch.bfloat16 else F32, B, H, n, d))


def diffattn_forward_host(q1, q2, k1, k2, v, lam, lambda_init_value: float, gamma=None, eps: float = 1e-5,
                          causal: bool = True, out=None, workspace=None, stream=None) -> torch.Tensor:
    """diffattn_forward on HOST tensors (page-locked for asynchronous copies).

    The library copies the inputs in, runs the forward and copies the output
    back, pipelined over chunks of the batch.  lam / gamma are device tensors
    (layer parameters); workspace is a device uint8 tensor of at least
    forward_host_workspace_bytes(...) bytes (allocated here if None).  The host
    output is complete once `stream` (default: the current stream) has
    reached this call.
    """
    B, n, H, d = q1.shape
    dt = q1.dtype
    for name, t in (("q1", q1), ("q2", q2), ("k1", k1), ("k2", k2)):
        _need_host(t, name, dt, (B, n, H, d))
    _need_host(v, "v", dt, (B, n, H, 2 * d))
    _need(lam, "lambda", torch.float32, (1,))
    if gamma is not None:
        _need(gamma, "gamma", torch.float32, (2 * d,))
    if out is None:
        out = torch.empty((B, n, H, 2 * d), dtype=dt).pin_memory()
    _need_host(out, "out", dt, (B, n, H, 2 * d))
    need = forward_host_workspace_bytes(dt, B, H, n, d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=lam.device)
    if not workspace.is_cuda or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must be a CUDA tensor of at least {need} bytes")
    _check(lib().diffattn_forward_host(_dt(q1), B, H, n, d, _ptr(q1), _ptr(q2), _ptr(k1), _ptr(k2), _ptr(v),
                                       _ptr(lam), float(lambda_init_value), _ptr(gamma), float(eps),
                                       1 if causal else 0, _ptr(out), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


def _ws_args(workspace, need):
    if workspace is None:
        return None, 0
    nbytes = workspace.numel() * workspace.element_size()
    if not workspace.is_cuda or nbytes < need:
        raise ValueError(f"workspace must be a CUDA tensor of at least {need} bytes")
    return _ptr(workspace), nbytes


def decode_workspace_bytes(B: int, H: int, d: int) -> int:
    """Device workspace that lets diffattn_decode split a (b, h) pair over several clusters."""
    return int(lib().diffattn_decode_workspace(B, H, d))


def v2_decode_workspace_bytes(B: int, Hq: int, d: int) -> int:
    return int(lib().diffattn_v2_decode_workspace(B, Hq, d))


def diffattn_decode(q1, q2, k1, k2, v, lam, lambda_init_value: float, gamma=None, eps: float = 1e-5,
                    lens=None, out=None, workspace=None, stream=None) -> torch.Tensor:
    """DIFF V1 decode: one new token per sequence over a key/value cache.

    q1, q2: [B, H, d]; k1, k2: [B, n, H, d]; v: [B, n, H, 2d] (bf16, d in
    {64, 128}); lens: int32 [B] visible keys per sequence or None (all n).
    workspace: None or a device tensor of decode_workspace_bytes(B, H, d)
    bytes (lets few (b, h) pairs use the whole GPU).  Returns out [B, H, 2d].
    """
    B, n, H, d = k1.shape
    dt = k1.dtype
    _need(q1, "q1", dt, (B, H, d))
    _need(q2, "q2", dt, (B, H, d))
    _need(k1, "k1", dt, (B, n, H, d))
    _need(k2, "k2", dt, (B, n, H, d))
    _need(v, "v", dt, (B, n, H, 2 * d))
    _need(lam, "lambda", torch.float32, (1,))
    if gamma is not None:
        _need(gamma, "gamma", torch.float32, (2 * d,))
    if lens is not None:
        _need(lens, "lens", torch.int32, (B,))
    if out is None:
        out = torch.empty((B, H, 2 * d), device=k1.device, dtype=dt)
    _need(out, "out", dt, (B, H, 2 * d))
    wp, wn = _ws_args(workspace, decode_workspace_bytes(B, H, d))
    _check(lib().diffattn_decode(_dt(k1), B, H, n, d, _ptr(q1), _ptr(q2), _ptr(k1), _ptr(k2), _ptr(v),
                                 _ptr(lens), _ptr(lam), float(lambda_init_value), _ptr(gamma), float(eps),
                                 _ptr(out), wp, wn, _stream(stream)))
    return out


def diffattn_decode_noalloc(q1, q2, k1, k2, v, lam, lambda_init_value: float, gamma=None, eps: float = 1e-5,
                            lens=None, out=None, stream=None) -> torch.Tensor:
    """diffattn_decode for callers that cannot allocate device memory.

    Same arguments and result as diffattn_decode with a workspace, but the
    split states live in a fixed 4 MiB scratch inside the library (B*H at
    most 504 pairs at d = 64, 254 at d = 128).  Calls that can overlap on the
    GPU share that scratch and must be serialised on one stream.  ``out`` is
    allocated here with torch when None; pass it to allocate nothing.
    """
    B, n, H, d = k1.shape
    dt = k1.dtype
    _need(q1, "q1", dt, (B, H, d))
    _need(q2, "q2", dt, (B, H, d))
    _need(k1, "k1", dt, (B, n, H, d))
    _need(k2, "k2", dt, (B, n, H, d))
    _need(v, "v", dt, (B, n, H, 2 * d))
    _need(lam, "lambda", torch.float32, (1,))
    if gamma is not None:
        _need(gamma, "gamma", torch.float32, (2 * d,))
    if lens is not None:
        _need(lens, "lens", torch.int32, (B,))
    if out is None:
        out = torch.empty((B, H, 2 * d), device=k1.device, dtype=dt)
    _need(out, "out", dt, (B, H, 2 * d))
    _check(lib().diffattn_decode_noalloc(_dt(k1), B, H, n, d, _ptr(q1), _ptr(q2), _ptr(k1), _ptr(k2), _ptr(v),
                                         _ptr(lens), _ptr(lam), float(lambda_init_value), _ptr(gamma), float(eps),
                                         _ptr(out), _stream(stream)))
    return out


def diffattn_v2_decode(q, k, v, lam_logits, lens=None, softmax_scale: float = 0.0, out=None,
                       workspace=None, stream=None) -> torch.Tensor:
    """DIFF V2 decode: one new token per sequence over a key/value cache.

    q: [B, Hq, d]; k, v: [B, n, Hkv, d] (bf16, d = 128); lam_logits: fp32
    [B, Hq/2] (one logit per pair of each sequence) or [Hq/2] (shared by all
    sequences); lens: int32 [B] or None.  Returns out [B, Hq/2, d].
    """
    B, n, Hkv, d = k.shape
    Hq = q.shape[1]
    dt = k.dtype
    _need(q, "q", dt, (B, Hq, d))
    _need(k, "k", dt, (B, n, Hkv, d))
    _need(v, "v", dt, (B, n, Hkv, d))
    if lam_logits.dim() == 1:
        _need(lam_logits, "lam_logits", torch.float32, (Hq // 2,))
        sb = 0
    else:
        _need(lam_logits, "lam_logits", torch.float32, (B, Hq // 2))
        sb = Hq // 2
    if lens is not None:
        _need(lens, "lens", torch.int32, (B,))
    if out is None:
        out = torch.empty((B, Hq // 2, d), device=k.device, dtype=dt)
    _need(out, "out", dt, (B, Hq // 2, d))
    wp, wn = _ws_args(workspace, v2_decode_workspace_bytes(B, Hq, d))
    _check(lib().diffattn_v2_decode(_dt(k), B, Hq, Hkv, n, d, _ptr(q), _ptr(k), _ptr(v), _ptr(lens),
                                    _ptr(lam_logits), sb, float(softmax_scale), _ptr(out), wp, wn,
                                    _stream(stream)))
    return out


def _need_fp8(t: torch.Tensor, name: str, shape):
    if t.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise ValueError(f"{name} must hold e4m3 bytes (torch.float8_e4m3fn or torch.uint8), got {t.dtype}")
    _need(t, name, None, shape)


def diffattn_decode_fp8k(q1, q2, k1, k2, k1_scale: float, k2_scale: float, v, lam, lambda_init_value: float,
                         gamma=None, eps: float = 1e-5, lens=None, out=None, workspace=None,
                         stream=None) -> torch.Tensor:
    """DIFF V1 decode over an FP8 key cache.

    k1, k2: [B, n, H, d] e4m3 codes (torch.float8_e4m3fn or their bytes as
    torch.uint8) of K_r / k_scale_r; the result is diffattn_decode's for the
    keys k_scale_r * k_r.  q1, q2, v, lam, gamma, lens, workspace: as for
    diffattn_decode (bf16, d in {64, 128}).  Returns out [B, H, 2d] (bf16).
    """
    B, n, H, d = k1.shape
    _need(q1, "q1", torch.bfloat16, (B, H, d))
    _need(q2, "q2", torch.bfloat16, (B, H, d))
    _need_fp8(k1, "k1", (B, n, H, d))
    _need_fp8(k2, "k2", (B, n, H, d))
    _need(v, "v", torch.bfloat16, (B, n, H, 2 * d))
    _need(lam, "lambda", torch.float32, (1,))
    if gamma is not None:
        _need(gamma, "gamma", torch.float32, (2 * d,))
    if lens is not None:
        _need(lens, "lens", torch.int32, (B,))
    if out is None:
        out = torch.empty((B, H, 2 * d), device=v.device, dtype=torch.bfloat16)
    _need(out, "out", torch.bfloat16, (B, H, 2 * d))
    wp, wn = _ws_args(workspace, decode_workspace_bytes(B, H, d))
    _check(lib().diffattn_decode_fp8k(B, H, n, d, _ptr(q1), _ptr(q2), _ptr(k1), _ptr(k2), float(k1_scale),
                                      float(k2_scale), _ptr(v), _ptr(lens), _ptr(lam), float(lambda_init_value),
                                      _ptr(gamma), float(eps), _ptr(out), wp, wn, _stream(stream)))
    return out


def diffattn_v2_decode_fp8k(q, k, k_scale: float, v, lam_logits, lens=None, softmax_scale: float = 0.0,
                            out=None, workspace=None, stream=None) -> torch.Tensor:
    """DIFF V2 decode over an FP8 key cache.

    k: [B, n, Hkv, d] e4m3 codes of K / k_scale (torch.float8_e4m3fn or
    torch.uint8); everything else as for diffattn_v2_decode (bf16, d = 128).
    Returns out [B, Hq/2, d] (bf16).
    """
    B, n, Hkv, d = k.shape
    Hq = q.shape[1]
    _need(q, "q", torch.bfloat16, (B, Hq, d))
    _need_fp8(k, "k", (B, n, Hkv, d))
    _need(v, "v", torch.bfloat16, (B, n, Hkv, d))
    if lam_logits.dim() == 1:
        _need(lam_logits, "lam_logits", torch.float32, (Hq // 2,))
        sb = 0
    else:
        _need(lam_logits, "lam_logits", torch.float32, (B, Hq // 2))
        sb = Hq // 2
    if lens is not None:
        _need(lens, "lens", torch.int32, (B,))
    if out is None:
        out = torch.empty((B, Hq // 2, d), device=v.device, dtype=torch.bfloat16)
    _need(out, "out", torch.bfloat16, (B, Hq // 2, d))
    wp, wn = _ws_args(workspace, v2_decode_workspace_bytes(B, Hq, d))
    _check(lib().diffattn_v2_decode_fp8k(B, Hq, Hkv, n, d, _ptr(q), _ptr(k), float(k_scale), _ptr(v), _ptr(lens),
                                         _ptr(lam_logits), sb, float(softmax_scale), _ptr(out), wp, wn,
                                         _stream(stream)))
    return out


def backward_workspace_bytes(B: int, H: int, n: int, d: int) -> int:
    """Device workspace diffattn_backward needs (per-row statistics, dO, dgamma shares)."""
    return int(lib().diffattn_backward_workspace(B, H, n, d))


def diffattn_backward(q1, q2, k1, k2, v, lam, lambda_init_value: float, dy, gamma=None, eps: float = 1e-5,
                      causal: bool = True, workspace=None, stream=None) -> dict:
    """DIFF V1 backward: gradients of diffattn_forward's output given dy.

    Shapes as for diffattn_forward; fp32 inputs (d <= 128, CUDA cores) or bf16
    inputs (d = 64, tensor cores); dy: [B, n, H, 2d] in the inputs' dtype.
    Returns a dict of fp32 gradients: dq1, dq2, dk1, dk2, dv (shaped like
    their inputs), dlam [1], dgamma [2d].  workspace: None (allocated here
    with torch) or a device tensor of backward_workspace_bytes(B, H, n, d) bytes.
    """
    B, n, H, d = q1.shape
    dt = q1.dtype
    for name, t, shp in (("q1", q1, (B, n, H, d)), ("q2", q2, (B, n, H, d)), ("k1", k1, (B, n, H, d)),
                         ("k2", k2, (B, n, H, d)), ("v", v, (B, n, H, 2 * d)), ("dy", dy, (B, n, H, 2 * d))):
        _need(t, name, dt, shp)
    _need(lam, "lambda", torch.float32, (1,))
    if gamma is not None:
        _need(gamma, "gamma", torch.float32, (2 * d,))
    need = backward_workspace_bytes(B, H, n, d)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q1.device)
    wp, wn = _ws_args(workspace, need)
    g = {k: torch.empty(t.shape, device=t.device, dtype=torch.float32)
         for k, t in (("dq1", q1), ("dq2", q2), ("dk1", k1), ("dk2", k2), ("dv", v))}
    g["dlam"] = torch.empty(1, device=q1.device, dtype=torch.float32)
    g["dgamma"] = torch.empty(2 * d, device=q1.device, dtype=torch.float32)
    _check(lib().diffattn_backward(_dt(q1), B, H, n, d, _ptr(q1), _ptr(q2), _ptr(k1), _ptr(k2), _ptr(v), _ptr(lam),
                                   float(lambda_init_value), _ptr(gamma), float(eps), 1 if causal else 0, _ptr(dy),
                                   _ptr(g["dq1"]), _ptr(g["dq2"]), _ptr(g["dk1"]), _ptr(g["dk2"]), _ptr(g["dv"]),
                                   _ptr(g["dlam"]), _ptr(g["dgamma"]), wp, wn, _stream(stream)))
    return g


def v2_backward_workspace_bytes(B: int, Hq: int, n: int, d: int) -> int:
    return int(lib().diffattn_v2_backward_workspace(B, Hq, n, d))


def diffattn_v2_backward(q, k, v, lam_logits, dy, causal: bool = True, softmax_scale: float = 0.0,
                         workspace=None, stream=None) -> dict:
    """DIFF V2 backward: gradients of diffattn_v2_forward's output given dy.

    q: [B, n, Hq, d]; k, v: [B, n, Hkv, d]; dy: [B, n, Hq/2, d], all fp32
    (d <= 128, CUDA cores) or all bf16 (d = 128, tensor cores); lam_logits:
    fp32 [B, n, Hq/2] (per token), [B, Hq/2] (per sequence) or [Hq/2] (per
    pair).  Returns a dict of fp32 gradients: dq, dk, dv and dlogits (shaped
    like lam_logits).
    """
    B, n, Hq, d = q.shape
    Hkv = k.shape[2]
    dt = q.dtype
    _need(q, "q", dt, (B, n, Hq, d))
    _need(k, "k", dt, (B, n, Hkv, d))
    _need(v, "v", dt, (B, n, Hkv, d))
    _need(dy, "dy", dt, (B, n, Hq // 2, d))
    G = Hq // 2
    f32 = torch.float32
    if lam_logits.dim() == 3:
        _need(lam_logits, "lam_logits", f32, (B, n, G))
        sb, st = n * G, G
    elif lam_logits.dim() == 2:
        _need(lam_logits, "lam_logits", f32, (B, G))
        sb, st = G, 0
    else:
        _need(lam_logits, "lam_logits", f32, (G,))
        sb, st = 0, 0
    need = v2_backward_workspace_bytes(B, Hq, n, d)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    wp, wn = _ws_args(workspace, need)
    g = {"dq": torch.empty(q.shape, device=q.device, dtype=f32), "dk": torch.empty(k.shape, device=q.device, dtype=f32),
         "dv": torch.empty(v.shape, device=q.device, dtype=f32), "dlogits": torch.empty_like(lam_logits)}
    _check(lib().diffattn_v2_backward(_dt(q), B, Hq, Hkv, n, d, _ptr(q), _ptr(k), _ptr(v), _ptr(lam_logits), sb, st,
                                      float(softmax_scale), 1 if causal else 0, _ptr(dy), _ptr(g["dq"]),
                                      _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["dlogits"]), wp, wn, _stream(stream)))
    return g


# ----------------------------------------------------------------------------- training pair
def forward_saved_bytes(B: int, H: int, n: int, d: int) -> int:
    """Device bytes that diffattn_forward_train saves for the backward (V1)."""
    return int(lib().diffattn_forward_saved_bytes(B, H, n, d))


def v2_forward_saved_bytes(B: int, Hq: int, n: int, d: int) -> int:
    """Device bytes that diffattn_v2_forward_train saves for the backward (V2)."""
    return int(lib().diffattn_v2_forward_saved_bytes(B, Hq, n, d))


def _saved_buf(saved, need, device):
    if saved is None:
        saved = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    if not saved.is_cuda or saved.dtype != torch.uint8 or saved.numel() < need:
        raise ValueError(f"saved must be a device uint8 tensor of at least {need} bytes")
    return saved


def diffattn_forward_train(q1, q2, k1, k2, v, lam, lambda_init_value: float, gamma=None, eps: float = 1e-5,
                           causal: bool = True, out=None, saved=None, stream=None):
    """diffattn_forward (bf16, d = 64) that also saves each row's lse and O_1, O_2 for
    diffattn_backward_saved.  Returns (out, saved)."""
    B, n, H, d = q1.shape
    for name, t, shp in (("q1", q1, (B, n, H, d)), ("q2", q2, (B, n, H, d)), ("k1", k1, (B, n, H, d)),
                         ("k2", k2, (B, n, H, d)), ("v", v, (B, n, H, 2 * d))):
        _need(t, name, torch.bfloat16, shp)
    _need(lam, "lambda", torch.float32, (1,))
    if gamma is not None:
        _need(gamma, "gamma", torch.float32, (2 * d,))
    if out is None:
        out = torch.empty((B, n, H, 2 * d), device=q1.device, dtype=torch.bfloat16)
    _need(out, "out", torch.bfloat16, (B, n, H, 2 * d))
    need = forward_saved_bytes(B, H, n, d)
    saved = _saved_buf(saved, need, q1.device)
    _check(lib().diffattn_forward_train(B, H, n, d, _ptr(q1), _ptr(q2), _ptr(k1), _ptr(k2), _ptr(v), _ptr(lam),
                                        float(lambda_init_value), _ptr(gamma), float(eps), 1 if causal else 0,
                                        _ptr(out), _ptr(saved), saved.numel(), _stream(stream)))
    return out, saved


def diffattn_backward_saved(q1, q2, k1, k2, v, lam, lambda_init_value: float, dy, saved, gamma=None,
                            eps: float = 1e-5, causal: bool = True, workspace=None, stream=None) -> dict:
    """diffattn_backward (bf16, d = 64) from the `saved` of diffattn_forward_train on the same inputs."""
    B, n, H, d = q1.shape
    for name, t, shp in (("q1", q1, (B, n, H, d)), ("q2", q2, (B, n, H, d)), ("k1", k1, (B, n, H, d)),
                         ("k2", k2, (B, n, H, d)), ("v", v, (B, n, H, 2 * d)), ("dy", dy, (B, n, H, 2 * d))):
        _need(t, name, torch.bfloat16, shp)
    _need(lam, "lambda", torch.float32, (1,))
    if gamma is not None:
        _need(gamma, "gamma", torch.float32, (2 * d,))
    need = backward_workspace_bytes(B, H, n, d)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q1.device)
    wp, wn = _ws_args(workspace, need)
    g = {k: torch.empty(t.shape, device=t.device, dtype=torch.float32)
         for k, t in (("dq1", q1), ("dq2", q2), ("dk1", k1), ("dk2", k2), ("dv", v))}
    g["dlam"] = torch.empty(1, device=q1.device, dtype=torch.float32)
    g["dgamma"] = torch.empty(2 * d, device=q1.device, dtype=torch.float32)
    _check(lib().diffattn_backward_saved(B, H, n, d, _ptr(q1), _ptr(q2), _ptr(k1), _ptr(k2), _ptr(v), _ptr(lam),
                                         float(lambda_init_value), _ptr(gamma), float(eps), 1 if causal else 0,
                                         _ptr(dy), _ptr(saved), saved.numel(), _ptr(g["dq1"]), _ptr(g["dq2"]),
                                         _ptr(g["dk1"]), _ptr(g["dk2"]), _ptr(g["dv"]), _ptr(g["dlam"]),
                                         _ptr(g["dgamma"]), wp, wn, _stream(stream)))
    return g


def _bwd_logit_strides(lam_logits, B, n, G):
    """Strides of the logits as the V2 backward takes them: [B, n, Hq/2], [B, Hq/2] or [Hq/2]."""
    f32 = torch.float32
    if lam_logits.dim() == 3:
        _need(lam_logits, "lam_logits", f32, (B, n, G))
        return n * G, G
    if lam_logits.dim() == 2:
        _need(lam_logits, "lam_logits", f32, (B, G))
        return G, 0
    _need(lam_logits, "lam_logits", f32, (G,))
    return 0, 0


def diffattn_v2_forward_train(q, k, v, lam_logits, causal: bool = True, softmax_scale: float = 0.0, out=None,
                              saved=None, stream=None):
    """diffattn_v2_forward (bf16, d = 128) that also saves each row's lse and O_1, O_2 for
    diffattn_v2_backward_saved; lam_logits [B, n, Hq/2], [B, Hq/2] or [Hq/2].  Returns (out, saved)."""
    B, n, Hq, d = q.shape
    Hkv = k.shape[2]
    _need(q, "q", torch.bfloat16, (B, n, Hq, d))
    _need(k, "k", torch.bfloat16, (B, n, Hkv, d))
    _need(v, "v", torch.bfloat16, (B, n, Hkv, d))
    G = Hq // 2
    sb, st = _bwd_logit_strides(lam_logits, B, n, G)
    if out is None:
        out = torch.empty((B, n, G, d), device=q.device, dtype=torch.bfloat16)
    _need(out, "out", torch.bfloat16, (B, n, G, d))
    need = v2_forward_saved_bytes(B, Hq, n, d)
    saved = _saved_buf(saved, need, q.device)
    _check(lib().diffattn_v2_forward_train(B, Hq, Hkv, n, d, _ptr(q), _ptr(k), _ptr(v), _ptr(lam_logits), sb, st,
                                           float(softmax_scale), 1 if causal else 0, _ptr(out), _ptr(saved),
                                           saved.numel(), _stream(stream)))
    return out, saved


def diffattn_v2_backward_saved(q, k, v, lam_logits, dy, saved, causal: bool = True, softmax_scale: float = 0.0,
                               workspace=None, stream=None) -> dict:
    """diffattn_v2_backward (bf16, d = 128) from the `saved` of diffattn_v2_forward_train on the same inputs."""
    B, n, Hq, d = q.shape
    Hkv = k.shape[2]
    for name, t, shp in (("q", q, (B, n, Hq, d)), ("k", k, (B, n, Hkv, d)), ("v", v, (B, n, Hkv, d)),
                         ("dy", dy, (B, n, Hq // 2, d))):
        _need(t, name, torch.bfloat16, shp)
    G = Hq // 2
    sb, st = _bwd_logit_strides(lam_logits, B, n, G)
    need = v2_backward_workspace_bytes(B, Hq, n, d)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    wp, wn = _ws_args(workspace, need)
    f32 = torch.float32
    g = {"dq": torch.empty(q.shape, device=q.device, dtype=f32), "dk": torch.empty(k.shape, device=q.device, dtype=f32),
         "dv": torch.empty(v.shape, device=q.device, dtype=f32), "dlogits": torch.empty_like(lam_logits)}
    _check(lib().diffattn_v2_backward_saved(B, Hq, Hkv, n, d, _ptr(q), _ptr(k), _ptr(v), _ptr(lam_logits), sb, st,
                                            float(softmax_scale), 1 if causal else 0, _ptr(dy), _ptr(saved),
                                            saved.numel(), _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]),
                                            _ptr(g["dlogits"]), wp, wn, _stream(stream)))
    return g


def lambda_reparam_backward(lq1, lk1, lq2, lk2, dlam, stream=None):
    """Gradients of lambda_reparam's lambda with respect to lq1, lk1, lq2, lk2, given dlam [1] (device)."""
    for name, t in (("lq1", lq1), ("lk1", lk1), ("lq2", lq2), ("lk2", lk2)):
        _need(t, name, torch.float32, (lq1.numel(),))
    _need(dlam, "dlam", torch.float32, (1,))
    outs = [torch.empty_like(t) for t in (lq1, lk1, lq2, lk2)]
    _check(lib().lambda_reparam_backward(_ptr(lq1), _ptr(lk1), _ptr(lq2), _ptr(lk2), lq1.numel(), _ptr(dlam),
                                         *(_ptr(o) for o in outs), _stream(stream)))
    return tuple(outs)


def _logit_strides(lam_logits, B, n, G):
    if lam_logits.shape == (G,):
        return 0, 0
    if lam_logits.shape == (n, G):
        return 0, G
    if lam_logits.shape == (B, n, G):
        return n * G, G
    raise ValueError(f"lam_logits must be [Hq/2], [n, Hq/2] or [B, n, Hq/2]; got {tuple(lam_logits.shape)}")


def diffattn_v2_forward_fp8qk(q, k, scales, v, lam_logits, causal: bool = True, softmax_scale: float = 0.0,
                              out=None, stream=None) -> torch.Tensor:
    """DIFF V2 forward with e4m3 queries and keys (QK^T on the FP8 tensor-core path).

    q: [B, n, Hq, 128], k: [B, n, Hkv, 128] e4m3 codes (torch.float8_e4m3fn or their bytes as uint8)
    of Q / q_scale and K / k_scale; scales = (q_scale, k_scale); v bf16 [B, n, Hkv, 128]; lam_logits
    as for diffattn_v2_forward.  The result is diffattn_v2_forward's for Q = q_scale e4m3(q),
    K = k_scale e4m3(k).  Returns out [B, n, Hq/2, 128] bf16.
    """
    B, n, Hq, d = q.shape
    Hkv = k.shape[2]
    _need_fp8(q, "q", (B, n, Hq, d))
    _need_fp8(k, "k", (B, n, Hkv, d))
    _need(v, "v", torch.bfloat16, (B, n, Hkv, d))
    G = Hq // 2
    _need(lam_logits, "lam_logits", torch.float32)
    sb, st = _logit_strides(lam_logits, B, n, G)
    if out is None:
        out = torch.empty((B, n, G, d), device=v.device, dtype=torch.bfloat16)
    _need(out, "out", torch.bfloat16, (B, n, G, d))
    qs, ks = (float(x) for x in scales)
    _check(lib().diffattn_v2_forward_fp8qk(B, Hq, Hkv, n, d, _ptr(q), _ptr(k), qs, ks, _ptr(v), _ptr(lam_logits),
                                           sb, st, float(softmax_scale), 1 if causal else 0, _ptr(out),
                                           _stream(stream)))
    return out


def diffattn_v2_forward(q, k, v, lam_logits, causal: bool = True, softmax_scale: float = 0.0, out=None,
                        stream=None) -> torch.Tensor:
    """DIFF V2 forward: out_g = attn[2g] - sigmoid(logit) attn[2g+1]; BSHD tensors.

    q: [B, n, Hq, d]; k, v: [B, n, Hkv, d]; lam_logits: fp32 [Hq/2] (one per
    pair), [n, Hq/2] or [B, n, Hq/2].  Returns out [B, n, Hq/2, d].
    """
    B, n, Hq, d = q.shape
    Hkv = k.shape[2]
    dt = q.dtype
    _need(q, "q", dt)
    _need(k, "k", dt, (B, n, Hkv, d))
    _need(v, "v", dt, (B, n, Hkv, d))
    G = Hq // 2
    _need(lam_logits, "lam_logits", torch.float32)
    sb, st = _logit_strides(lam_logits, B, n, G)
    if out is None:
        out = torch.empty((B, n, G, d), device=q.device, dtype=dt)
    _need(out, "out", dt, (B, n, G, d))
    _check(lib().diffattn_v2_forward(_dt(q), B, Hq, Hkv, n, d, _ptr(q), _ptr(k), _ptr(v), _ptr(lam_logits),
                                     sb, st, float(softmax_scale), 1 if causal else 0, _ptr(out),
                                     _stream(stream)))
    return out


def projection(a, w, out=None, stream=None) -> torch.Tensor:
    """out = a w^T on the tensor cores: a [M, K], w [N, K] (bf16; K, N multiples of 8) -> [M, N] bf16."""
    M, K = a.shape
    N = w.shape[0]
    _need(a, "a", torch.bfloat16, (M, K))
    _need(w, "w", torch.bfloat16, (N, K))
    if out is None:
        out = torch.empty((M, N), device=a.device, dtype=torch.bfloat16)
    _need(out, "out", torch.bfloat16, (M, N))
    _check(lib().diffattn_projection(M, N, K, _ptr(a), _ptr(w), _ptr(out), _stream(stream)))
    return out


def layer_workspace_bytes(B: int, n: int, H: int, d: int) -> int:
    return int(lib().diffattn_layer_workspace(B, n, H, d))


def layer_forward(x, w_qkv, w_o, lq1, lk1, lq2, lk2, lambda_init_value: float, H: int, gamma=None,
                  eps: float = 1e-5, causal: bool = True, out=None, workspace=None, stream=None) -> torch.Tensor:
    """DIFF V1 attention layer: X [W^Q | W^K | W^V], the operator with the per-head norm, W^O.

    x: [B, n, D] bf16; w_qkv: [3 H 2d, D] bf16 (rows: W^Q's columns, then W^K's, then W^V's; head i's
    2d columns of W^Q hold Q_1 then Q_2); w_o: [D, H 2d] bf16; lq1..lk2: fp32 [d]; gamma: fp32 [2d] or
    None.  workspace: a device tensor of layer_workspace_bytes(B, n, H, d) bytes (allocated here if
    None).  Returns out [B, n, D] bf16.
    """
    B, n, D = x.shape
    d = w_qkv.shape[0] // (6 * H)
    _need(x, "x", torch.bfloat16, (B, n, D))
    _need(w_qkv, "w_qkv", torch.bfloat16, (6 * H * d, D))
    _need(w_o, "w_o", torch.bfloat16, (D, 2 * H * d))
    for name, t in (("lq1", lq1), ("lk1", lk1), ("lq2", lq2), ("lk2", lk2)):
        _need(t, name, torch.float32, (d,))
    if gamma is not None:
        _need(gamma, "gamma", torch.float32, (2 * d,))
    if out is None:
        out = torch.empty((B, n, D), device=x.device, dtype=torch.bfloat16)
    _need(out, "out", torch.bfloat16, (B, n, D))
    need = layer_workspace_bytes(B, n, H, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
    wp, wn = _ws_args(workspace, need)
    _check(lib().diffattn_layer_forward(B, n, D, H, d, _ptr(x), _ptr(w_qkv), _ptr(w_o), _ptr(lq1), _ptr(lk1),
                                        _ptr(lq2), _ptr(lk2), float(lambda_init_value), _ptr(gamma), float(eps),
                                        1 if causal else 0, _ptr(out), wp, wn, _stream(stream)))
    return out


def v2_layer_workspace_bytes(B: int, n: int, Hq: int, Hkv: int, d: int) -> int:
    return int(lib().diffattn_v2_layer_workspace(B, n, Hq, Hkv, d))


def v2_layer_forward(x, w_qkvl, w_o, Hq: int, Hkv: int, causal: bool = True, out=None, workspace=None,
                     stream=None) -> torch.Tensor:
    """DIFF V2 attention layer: X [W^Q | W^K | W^V | W^lambda], the V2 operator, W^O.

    x: [B, n, D] bf16; w_qkvl: [(Hq + 2 Hkv) d + Hq/2, D] bf16 (rows: W^Q's columns, W^K's, W^V's,
    then the Hq/2 pair-logit columns of W^lambda); w_o: [D, Hq/2 d] bf16.  Returns out [B, n, D].
    """
    B, n, D = x.shape
    G = Hq // 2
    d = (w_qkvl.shape[0] - G) // (Hq + 2 * Hkv)
    _need(x, "x", torch.bfloat16, (B, n, D))
    _need(w_qkvl, "w_qkvl", torch.bfloat16, ((Hq + 2 * Hkv) * d + G, D))
    _need(w_o, "w_o", torch.bfloat16, (D, G * d))
    if out is None:
        out = torch.empty((B, n, D), device=x.device, dtype=torch.bfloat16)
    _need(out, "out", torch.bfloat16, (B, n, D))
    need = v2_layer_workspace_bytes(B, n, Hq, Hkv, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
    wp, wn = _ws_args(workspace, need)
    _check(lib().diffattn_v2_layer_forward(B, n, D, Hq, Hkv, d, _ptr(x), _ptr(w_qkvl), _ptr(w_o),
                                           1 if causal else 0, _ptr(out), wp, wn, _stream(stream)))
    return out


# ----------------------------------------------------------------------------- positions and caches
class RopeSpec(ctypes.Structure):
    """A rotation, as rope_spec or rope_from_frequencies makes it."""
    _fields_ = [("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("mult", ctypes.c_float),
                ("turns", ctypes.c_ulonglong * 64)]


class _SharedRopeSpec(RopeSpec):
    """What rope_spec hands to every caller of the same arguments: its fields cannot be set."""

    def __setattr__(self, name, value):
        raise AttributeError("rope_spec's rotations are shared; RopeSpec.from_buffer_copy(spec) is one to change")

    @property
    def turns(self):
        return RopeSpec.turns.__get__(self)[:]


ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


@functools.lru_cache(maxsize=256)
def rope_spec(rot_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "none",
              factor: float = 1.0, original_context: int = 0, beta_fast: float = 32.0,
              beta_slow: float = 1.0) -> RopeSpec:
    """Rotary positions on the first rot_dim channels of a head: theta_i = base^(-2i / rot_dim), scaled.

    interleaved: pairs (2i, 2i + 1) instead of (i, i + rot_dim / 2).  scaling: "none", "linear"
    (theta / factor), "ntk" (base factor^(rot_dim / (rot_dim - 2))) or "yarn" (between the two, by the
    turns a pair makes over original_context positions; the rotated values times 0.1 ln(factor) + 1).
    Host only.  The same arguments give the same object, which cannot be changed.
    """
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
    spec = RopeSpec()
    _check(lib().diffattn_rope_init(ctypes.byref(spec), rot_dim, 1 if interleaved else 0, base, ROPE_SCALINGS[scaling],
                                    factor, original_context, beta_fast, beta_slow))
    return _SharedRopeSpec.from_buffer_copy(spec)


def rope_from_frequencies(frequencies, interleaved: bool = False, mult: float = 1.0) -> RopeSpec:
    """A rotation of 2 len(frequencies) channels by frequencies of the caller's own (radians per position)."""
    fr = [float(x) for x in frequencies]
    spec = RopeSpec()
    _check(lib().diffattn_rope_from_frequencies(ctypes.byref(spec), 2 * len(fr), 1 if interleaved else 0,
                                                (ctypes.c_double * max(1, len(fr)))(*fr), mult))
    return spec


def _on(t, name, dtype, shape, dev):
    """_need, on the device `dev` (an index), which has to be the current one."""
    if t.dtype != dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        _need(t, name, dtype, shape)
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on device {dev}, got {t.device}")


def _current(t, name) -> int:
    """The device index of t, which has to be the current device."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    dev = t.get_device()
    if dev != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    return dev


_PTRS = [ctypes.c_void_p * k for k in range(5)]
_INTS = [ctypes.c_int * k for k in range(5)]


def _empty(shape, dtype, device, stream):
    """torch.empty for a kernel on `stream`: memory of that stream's own, as under torch.cuda.stream(stream)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _like(x, stream):
    return torch.empty_like(x) if stream is None else _empty(x.shape, x.dtype, x.device, stream)


def rope(tensors, spec: RopeSpec, positions=None, inverse: bool = False, out=None, stream=None) -> list:
    """Rotary positions on up to four tensors [B, n, heads, d] (bf16 or fp32, d <= 128) in one kernel.

    positions: int32 [B, n] or None (token t at position t).  inverse: the rotation by the negative
    angles, which is also the backward pass: the gradients of the unrotated tensors from those of the
    rotated ones.  out: None or tensors like the inputs, each allowed to be its own input (in place).
    Returns the list of rotated tensors.
    """
    xs = list(tensors)
    if not xs:
        return []
    if len(xs) > 4:
        raise ValueError(f"at most 4 tensors a call, got {len(xs)}")
    dev = _current(xs[0], "tensors[0]")
    B, n, _, d = xs[0].shape
    dt = xs[0].dtype
    for k, x in enumerate(xs):
        _on(x, f"tensors[{k}]", dt, (B, n, x.shape[2] if x.dim() == 4 else -1, d), dev)
    if positions is not None:
        _on(positions, "positions", torch.int32, (B, n), dev)
    if out is None:
        out = [_like(x, stream) for x in xs]
    else:
        out = list(out)
        if len(out) != len(xs):
            raise ValueError(f"out must hold {len(xs)} tensors, got {len(out)}")
        for k, (x, o) in enumerate(zip(xs, out)):
            _on(o, f"out[{k}]", dt, x.shape, dev)
    m = len(xs)
    _check(lib().diffattn_rope(_dt(xs[0]), B, n, d, m, _PTRS[m](*[x.data_ptr() for x in xs]),
                               _INTS[m](*[x.shape[2] for x in xs]), ctypes.byref(spec), _addr(positions),
                               1 if inverse else 0, _PTRS[m](*[o.data_ptr() for o in out]), _stream(stream)))
    return out


CACHE_FORMATS = {"bf16": 0, "fp8k": 1, "fp8": 2}
_CODES = (torch.float8_e4m3fn, torch.uint8)


class KVCache:
    """A key/value cache: V1 (k1, k2 [B, n, H, d], v [B, n, H, 2d]) or, with k2 None, V2 (k1, v [B, n, Hkv, d]).

    fmt: "bf16"; "fp8k" (e4m3 keys, one scale a tensor: k1_scale, k2_scale; bf16 values); "fp8" (e4m3
    keys and values, fp32 scales a row: k1_scales, k2_scales, v_scales [B, H, n]).  e4m3 tensors are
    torch.float8_e4m3fn or their bytes as torch.uint8.  cache_v1 and cache_v2 allocate one.  A tensor may
    be replaced by one of the same type, shape and device, a key scale by another number; the rest is fixed.
    """

    __slots__ = ("_fmt", "_code", "_k1", "_k2", "_v", "k1_scale", "k2_scale", "_k1_scales", "_k2_scales", "_v_scales",
                 "_B", "_n", "_H", "_d", "_dev")

    def __init__(self, fmt, k1, k2, v, k1_scale: float = 1.0, k2_scale: float = 1.0, k1_scales=None, k2_scales=None,
                 v_scales=None):
        if fmt not in CACHE_FORMATS:
            raise ValueError(f"the cache format must be one of {sorted(CACHE_FORMATS)}, got {fmt!r}")
        if not k1.is_cuda:
            raise ValueError("k1 must be a CUDA tensor")
        B, n, H, d = k1.shape
        dev = k1.get_device()
        kt, vt = (torch.bfloat16 if fmt == "bf16" else k1.dtype), (v.dtype if fmt == "fp8" else torch.bfloat16)
        if (fmt != "bf16" and kt not in _CODES) or (fmt == "fp8" and vt not in _CODES):
            raise ValueError("e4m3 tensors must be torch.float8_e4m3fn or torch.uint8")
        _on(k1, "k1", kt, (B, n, H, d), dev)
        if k2 is not None:
            _on(k2, "k2", kt, (B, n, H, d), dev)
        _on(v, "v", vt, (B, n, H, d if k2 is None else 2 * d), dev)
        if fmt == "fp8":
            for name, x, want in (("k1_scales", k1_scales, True), ("k2_scales", k2_scales, k2 is not None),
                                  ("v_scales", v_scales, True)):
                if want:
                    if x is None:
                        raise ValueError(f"an fp8 cache needs {name}")
                    _on(x, name, torch.float32, (B, H, n), dev)
        self._fmt, self._code = fmt, CACHE_FORMATS[fmt]
        self._B, self._n, self._H, self._d, self._dev = B, n, H, d, dev
        self._k1, self._k2, self._v = k1, k2, v
        self.k1_scale, self.k2_scale = float(k1_scale), float(k2_scale)
        self._k1_scales, self._k2_scales, self._v_scales = k1_scales, k2_scales, v_scales


def _replaceable(name):
    """A cache's tensor, to be replaced by its like alone: the calls take the shapes for checked."""
    def put(self, x):
        old = getattr(self, "_" + name)
        if old is None:
            raise AttributeError(f"this cache has no {name}")
        _on(x, name, old.dtype, old.shape, self._dev)
        setattr(self, "_" + name, x)
    return property(operator.attrgetter("_" + name), put)


for _name in ("k1", "k2", "v", "k1_scales", "k2_scales", "v_scales"):
    setattr(KVCache, _name, _replaceable(_name))
for _name in ("fmt", "code", "B", "n", "H", "d", "dev"):
    setattr(KVCache, _name, property(operator.attrgetter("_" + _name)))
del _name


def _new_cache(B, n, H, d, dv, two, fmt, device, scales):
    if fmt not in CACHE_FORMATS:
        raise ValueError(f"the cache format must be one of {sorted(CACHE_FORMATS)}, got {fmt!r}")
    kt = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
    vt = torch.float8_e4m3fn if fmt == "fp8" else torch.bfloat16

    def sc(want=True):
        return torch.zeros((B, H, n), device=device, dtype=torch.float32) if fmt == "fp8" and want else None
    return KVCache(fmt, torch.zeros((B, n, H, d), device=device, dtype=kt),
                   torch.zeros((B, n, H, d), device=device, dtype=kt) if two else None,
                   torch.zeros((B, n, H, dv), device=device, dtype=vt), *scales, sc(), sc(two), sc())


def cache_v1(B: int, n: int, H: int, d: int, fmt: str = "bf16", device="cuda", k1_scale: float = 1.0,
             k2_scale: float = 1.0) -> KVCache:
    """An empty V1 cache of n tokens a sequence."""
    return _new_cache(B, n, H, d, 2 * d, True, fmt, device, (k1_scale, k2_scale))


def cache_v2(B: int, n: int, Hkv: int, d: int, fmt: str = "bf16", device="cuda", k_scale: float = 1.0) -> KVCache:
    """An empty V2 cache of n tokens a sequence."""
    return _new_cache(B, n, Hkv, d, d, False, fmt, device, (k_scale, 1.0))


def _need_kind(cache, two):
    if (cache._k2 is not None) != two:
        raise ValueError("a V1 cache (k1 and k2) is needed" if two else "a V2 cache (one key tensor) is needed")
    if cache._dev != torch.cuda.current_device():
        raise ValueError(f"the cache is on device {cache._dev}, the current device is {torch.cuda.current_device()}")


def _int32(t, name, shape, dev):
    if t is None:
        return None
    _on(t, name, torch.int32, shape, dev)
    return t.data_ptr()


def _addr(t):
    return None if t is None else t.data_ptr()


def cache_append(cache: KVCache, k1, k2, v, q1=None, q2=None, rope=None, positions=None, lens=None, ntok=None,
                 q1_out=None, q2_out=None, stream=None):
    """Write T new tokens a sequence into a V1 cache: keys rotated and quantised, values quantised, queries rotated.

    k1, k2 (and q1, q2, or both None): bf16 [B, T, H, d]; v: [B, T, H, 2d].  rope: a RopeSpec or None;
    positions: int32 [B, T] or None (the cache row).  lens: int32 [B], the first row written (None: 0);
    ntok: int32 [B] tokens a sequence (None: T; later ones leave the cache as it is and give zero
    queries).  Returns (q1_out, q2_out), the rotated queries (None without queries).
    """
    _need_kind(cache, True)
    B, T, H, d = k1.shape
    dev, bf = cache._dev, torch.bfloat16
    if (B, H, d) != (cache._B, cache._H, cache._d):
        raise ValueError(f"keys {tuple(k1.shape)} do not fit a cache of B={cache._B}, H={cache._H}, d={cache._d}")
    shp = (B, T, H, d)
    _on(k1, "k1", bf, shp, dev)
    _on(k2, "k2", bf, shp, dev)
    _on(v, "v", bf, (B, T, H, 2 * d), dev)
    if (q1 is None) != (q2 is None):
        raise ValueError("q1 and q2 come together")
    if q1 is not None:
        _on(q1, "q1", bf, shp, dev)
        _on(q2, "q2", bf, shp, dev)
        q1_out = _like(q1, stream) if q1_out is None else q1_out
        q2_out = _like(q2, stream) if q2_out is None else q2_out
        _on(q1_out, "q1_out", bf, shp, dev)
        _on(q2_out, "q2_out", bf, shp, dev)
    _check(lib().diffattn_cache_append(
        cache._code, B, T, H, cache._n, d, _addr(q1), _addr(q2), k1.data_ptr(), k2.data_ptr(), v.data_ptr(),
        None if rope is None else ctypes.byref(rope), _int32(positions, "positions", (B, T), dev),
        _int32(lens, "lens", (B,), dev), _int32(ntok, "ntok", (B,), dev), _addr(q1_out), _addr(q2_out),
        cache._k1.data_ptr(), cache._k2.data_ptr(), cache._v.data_ptr(), cache.k1_scale, cache.k2_scale,
        _addr(cache._k1_scales), _addr(cache._k2_scales), _addr(cache._v_scales), _stream(stream)))
    return None if q1 is None else (q1_out, q2_out)


def v2_cache_append(cache: KVCache, k, v, q=None, rope=None, positions=None, lens=None, ntok=None, q_out=None,
                    stream=None):
    """cache_append for a V2 cache: k, v bf16 [B, T, Hkv, d]; q [B, T, Hq, d] or None.  Returns q_out."""
    _need_kind(cache, False)
    B, T, H, d = k.shape
    dev, bf = cache._dev, torch.bfloat16
    if (B, H, d) != (cache._B, cache._H, cache._d):
        raise ValueError(f"keys {tuple(k.shape)} do not fit a cache of B={cache._B}, Hkv={cache._H}, d={cache._d}")
    _on(k, "k", bf, (B, T, H, d), dev)
    _on(v, "v", bf, (B, T, H, d), dev)
    Hq = 0
    if q is not None:
        Hq = q.shape[2]
        _on(q, "q", bf, (B, T, Hq, d), dev)
        q_out = _like(q, stream) if q_out is None else q_out
        _on(q_out, "q_out", bf, (B, T, Hq, d), dev)
    _check(lib().diffattn_v2_cache_append(
        cache._code, B, T, Hq, H, cache._n, d, _addr(q), k.data_ptr(), v.data_ptr(),
        None if rope is None else ctypes.byref(rope), _int32(positions, "positions", (B, T), dev),
        _int32(lens, "lens", (B,), dev), _int32(ntok, "ntok", (B,), dev), _addr(q_out), cache._k1.data_ptr(),
        cache._v.data_ptr(), cache.k1_scale, _addr(cache._k1_scales), _addr(cache._v_scales), _stream(stream)))
    return None if q is None else q_out


def cache_keep(cache: KVCache, lens, path, nkeep, new_lens=None, stream=None) -> torch.Tensor:
    """Move the rows of each accepted path's nodes to the front of the drafted rows, in place.

    Row lens[b] + path[b, i] moves to row lens[b] + i for i < nkeep[b]; path: int32 [B, A], ascending
    node numbers, A <= 64; lens, nkeep: int32 [B].  Works on V1 and V2 caches.  Returns new_lens,
    int32 [B]: lens plus the nodes kept.
    """
    _need_kind(cache, cache._k2 is not None)
    B, dev = cache._B, cache._dev
    if path.dim() != 2:
        raise ValueError(f"path must be [B, A], got {tuple(path.shape)}")
    A = path.shape[1]
    if new_lens is None:
        new_lens = _like(lens, stream)
    a = (_int32(lens, "lens", (B,), dev), _int32(path, "path", (B, A), dev), _int32(nkeep, "nkeep", (B,), dev),
         _int32(new_lens, "new_lens", (B,), dev), _stream(stream))
    if cache._k2 is not None:
        _check(lib().diffattn_cache_keep(
            cache._code, B, A, cache._H, cache._n, cache._d, cache._k1.data_ptr(), cache._k2.data_ptr(), cache._v.data_ptr(),
            _addr(cache._k1_scales), _addr(cache._k2_scales), _addr(cache._v_scales), *a))
    else:
        _check(lib().diffattn_v2_cache_keep(
            cache._code, B, A, cache._H, cache._n, cache._d, cache._k1.data_ptr(), cache._v.data_ptr(),
            _addr(cache._k1_scales), _addr(cache._v_scales), *a))
    return new_lens


@functools.lru_cache(maxsize=256)
def tree_decode_workspace_bytes(B: int, T: int, H: int, d: int) -> int:
    """Device workspace of tree_decode (partial softmax states)."""
    return int(lib().diffattn_tree_decode_workspace(B, T, H, d))


@functools.lru_cache(maxsize=256)
def v2_tree_decode_workspace_bytes(B: int, T: int, Hq: int, Hkv: int, d: int) -> int:
    return int(lib().diffattn_v2_tree_decode_workspace(B, T, Hq, Hkv, d))


def _tree_args(lens, ntok, mask, B, T, dev):
    sb = 0
    if mask is not None:
        if mask.dim() == 2:
            _on(mask, "mask", torch.int64, (B, T), dev)
            sb = T
        else:
            _on(mask, "mask", torch.int64, (T,), dev)
    return _int32(lens, "lens", (B,), dev), _int32(ntok, "ntok", (B,), dev), _addr(mask), sb


def _tree_workspace(workspace, need, dev, like, stream):
    if workspace is None:
        return _empty((max(need, 16),), torch.uint8, like.device, stream)
    if not workspace.is_contiguous() or workspace.get_device() != dev:
        raise ValueError(f"workspace must be contiguous and on device {dev}")
    return workspace


def tree_decode(q1, q2, cache: KVCache, lam, lambda_init_value: float, gamma=None, eps: float = 1e-5, lens=None,
                ntok=None, mask=None, out=None, workspace=None, stream=None) -> torch.Tensor:
    """DIFF V1 attention of T <= 64 drafted tokens a sequence over a cache that already holds their keys and values.

    q1, q2: bf16 [B, T, H, d].  lens: int32 [B] keys before the drafts (None: n - T), which every
    token sees; the drafts are rows lens[b] .. lens[b] + ntok[b] - 1 (ntok: int32 [B] or None: T).
    mask: int64 words [B, T] or [T], bit u of word t: token t sees draft u; None: a chain (u <= t).
    T = 1 is a plain decode step.  lam, gamma, eps: as for diffattn_decode.  workspace: a device tensor
    of tree_decode_workspace_bytes(B, T, H, d) bytes (allocated here if None).  Returns out
    [B, T, H, 2d] bf16; tokens from ntok[b] on, and tokens that see nothing, are zeros.
    """
    _need_kind(cache, True)
    B, T, H, d = q1.shape
    dev, bf = cache._dev, torch.bfloat16
    if (B, H, d) != (cache._B, cache._H, cache._d):
        raise ValueError(f"queries {tuple(q1.shape)} do not fit a cache of B={cache._B}, H={cache._H}, d={cache._d}")
    _on(q1, "q1", bf, (B, T, H, d), dev)
    _on(q2, "q2", bf, (B, T, H, d), dev)
    _on(lam, "lambda", torch.float32, (1,), dev)
    if gamma is not None:
        _on(gamma, "gamma", torch.float32, (2 * d,), dev)
    a = _tree_args(lens, ntok, mask, B, T, dev)
    if out is None:
        out = _empty((B, T, H, 2 * d), bf, q1.device, stream)
    _on(out, "out", bf, (B, T, H, 2 * d), dev)
    need = tree_decode_workspace_bytes(B, T, H, d)
    workspace = _tree_workspace(workspace, need, dev, q1, stream)  # (alive until the kernels are in their stream)
    wp, wn = _ws_args(workspace, need)
    _check(lib().diffattn_tree_decode(
        cache._code, B, T, H, cache._n, d, q1.data_ptr(), q2.data_ptr(), cache._k1.data_ptr(), cache._k2.data_ptr(),
        cache.k1_scale, cache.k2_scale, _addr(cache._k1_scales), _addr(cache._k2_scales), cache._v.data_ptr(),
        _addr(cache._v_scales), *a, lam.data_ptr(), lambda_init_value, _addr(gamma), eps, out.data_ptr(), wp, wn,
        _stream(stream)))
    return out


def v2_tree_decode(q, cache: KVCache, lam_logits, lens=None, ntok=None, mask=None, softmax_scale: float = 0.0,
                   out=None, workspace=None, stream=None) -> torch.Tensor:
    """tree_decode for DIFF V2: q bf16 [B, T, Hq, d]; lam_logits fp32 [B, T, Hq/2], [B, Hq/2] or [Hq/2].

    workspace: v2_tree_decode_workspace_bytes(B, T, Hq, Hkv, d) bytes.  Returns out [B, T, Hq/2, d].
    """
    _need_kind(cache, False)
    B, T, Hq, d = q.shape
    dev, bf, G = cache._dev, torch.bfloat16, Hq // 2
    if (B, d) != (cache._B, cache._d):
        raise ValueError(f"queries {tuple(q.shape)} do not fit a cache of B={cache._B}, d={cache._d}")
    _on(q, "q", bf, (B, T, Hq, d), dev)
    sb, st = (T * G, G) if lam_logits.dim() == 3 else (G, 0) if lam_logits.dim() == 2 else (0, 0)
    _on(lam_logits, "lam_logits", torch.float32, ((B, T, G), (B, G), (G,))[3 - lam_logits.dim()]
        if 1 <= lam_logits.dim() <= 3 else (B, T, G), dev)
    a = _tree_args(lens, ntok, mask, B, T, dev)
    if out is None:
        out = _empty((B, T, G, d), bf, q.device, stream)
    _on(out, "out", bf, (B, T, G, d), dev)
    need = v2_tree_decode_workspace_bytes(B, T, Hq, cache._H, d)
    workspace = _tree_workspace(workspace, need, dev, q, stream)
    wp, wn = _ws_args(workspace, need)
    _check(lib().diffattn_v2_tree_decode(
        cache._code, B, T, Hq, cache._H, cache._n, d, q.data_ptr(), cache._k1.data_ptr(), cache.k1_scale,
        _addr(cache._k1_scales), cache._v.data_ptr(), _addr(cache._v_scales), *a, lam_logits.data_ptr(), sb, st,
        float(softmax_scale), out.data_ptr(), wp, wn, _stream(stream)))
    return out


# ----------------------------------------------------------------------------- the block around the layer
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


def _act_code(act: str) -> int:
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError(f"the activation must be one of {sorted(ACTIVATIONS)}, got {act!r}")
    return code


def _rows(t, name, dtype, shape, dev):
    """The row stride (elements) of a tensor [..., width]: contiguous, or 2-D with contiguous rows."""
    if t.dtype == dtype and t.shape == shape and t.is_cuda and t.get_device() == dev:
        if t.is_contiguous():
            return shape[-1]
        if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= shape[1]:
            return t.stride(0)
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on device {dev}, got {t.device}")
    raise ValueError(f"{name} must be contiguous, or 2-D with contiguous rows that do not overlap")


_bf16, _f32 = torch.bfloat16, torch.float32


def _here(dev, stream) -> int:
    """The raw stream `stream` (None: the current one) of the current device, which has to be `dev`."""
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"tensors are on device {dev}, the current device is cuda:{torch._C._cuda_getDevice()}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError(f"tensors are on device {dev}, the stream is on device {stream.device_index}")
    return stream.cuda_stream


def _product(x, w, name, wname):
    """Of rows x [..., K] under weights w [n, K]: device, n, K, the leading shape, the number of rows, the row stride."""
    dev = x.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape, wshape = x.shape, w.shape
    if len(wshape) != 2 or not shape:
        raise ValueError(f"{name} must be [..., K] and {wname} [n, K]")
    n, K = wshape
    lead = shape[:-1]
    M = lead.numel()
    if (M | n | K) >> 31:
        raise ValueError(f"{name} {tuple(shape)} and {wname} {tuple(wshape)}: sizes are below 2^31")
    if w.dtype is not _bf16 or w.get_device() != dev or not w.is_contiguous():
        _on(w, wname, _bf16, wshape, dev)
    if x.dtype is _bf16 and shape[-1] == K and x.is_contiguous():
        return dev, n, K, lead, M, K
    return dev, n, K, lead, M, _rows(x, name, _bf16, lead + (K,), dev)


def _linear(a, w, bias, act, residual, dtype, out, pre, stream):
    dev, N, K, lead, M, lda = _product(a, w, "a", "w")
    raw = _here(dev, stream)
    shape = lead + (N,)
    ldo = ldr = N
    if out is None:
        if dtype is None:
            dtype = _bf16
        out = torch.empty(shape, dtype=dtype, device=a.device) if stream is None else _empty(shape, dtype, a.device, stream)
    else:
        if dtype is not None and out.dtype is not dtype:
            raise ValueError(f"out must be {dtype}, got {out.dtype}")
        dtype = out.dtype
        ldo = _rows(out, "out", dtype, shape, dev)
    code = ACTIVATIONS.get(act)
    if code is None:
        code = _act_code(act)
    if bias is not None:
        _on(bias, "bias", _f32, (N,), dev)
        bias = bias.data_ptr()
    if residual is not None:
        if residual.dtype is not dtype or residual.shape != shape or residual.get_device() != dev or not residual.is_contiguous():
            ldr = _rows(residual, "residual", dtype, shape, dev)
        residual = residual.data_ptr()
    if pre is not None:
        _on(pre, "pre", _bf16, shape, dev)
        pre = pre.data_ptr()
    st = lib().diffattn_linear(M, N, K, a.data_ptr(), lda, w.data_ptr(), bias, code, residual, ldr,
                               BF16 if dtype is _bf16 else _dt(out), out.data_ptr(), ldo, pre, raw)
    if st:
        _check(st)
    return out


def linear(a, w, bias=None, act: str = "none", residual=None, dtype=None, out=None, stream=None) -> torch.Tensor:
    """out = residual + act(a w^T + bias) in one kernel: a [..., K], w [N, K] (bf16; N, K multiples of 8).

    bias: fp32 [N]; act: "none", "relu", "gelu", "gelu_tanh" or "silu"; residual: [..., N] of the output's
    type, and may be out itself; dtype: bf16 (default) or fp32.  a, residual and out may be 2-D with rows
    further apart (multiples of 8 elements; fp32: of 4), e.g. columns of a wider tensor.
    """
    return _linear(a, w, bias, act, residual, dtype, out, None, stream)


def linear_train(a, w, bias=None, act: str = "none", residual=None, dtype=None, out=None, pre=None, stream=None):
    """linear that also keeps a w^T + bias (bf16) for linear_backward: returns (out, pre)."""
    if pre is None:
        pre = _empty(a.shape[:-1] + w.shape[:1], torch.bfloat16, a.device, stream)
    return _linear(a, w, bias, act, residual, dtype, out, pre, stream), pre


@functools.lru_cache(maxsize=1024)
def linear_backward_workspace_bytes(M: int, N: int, K: int, act: str | None = None, bias: bool = True) -> int:
    """Workspace of linear_backward; act=None: enough for any activation.  Without one only the bias gradient needs any."""
    if act is None:
        return int(lib().diffattn_linear_backward_workspace(M, N, K))
    return int(lib().diffattn_linear_backward_workspace_for(M, N, K, _act_code(act), 1 if bias else 0))


def _workspace(workspace, need, dev, like, stream):
    if workspace is None:
        return _empty((need,), torch.uint8, like.device, stream) if need else None
    if not workspace.is_cuda or workspace.get_device() != dev or not workspace.is_contiguous() or workspace.nbytes < need:
        raise ValueError(f"workspace must be a contiguous CUDA tensor of at least {need} bytes on device {dev}")
    return workspace


def _grads(out, wanted, dev, device, stream) -> dict:
    """Tensors for the gradients `wanted` ((name, shape, dtype), ...): the caller's in the dict `out`, or new ones."""
    if out is None and stream is None:
        empty = torch.empty
        return {name: empty(shape, dtype=dtype, device=device) for name, shape, dtype in wanted}
    r, out = {}, out or {}
    known = [name for name, _, _ in wanted]
    for k in out:
        if k not in known:
            raise ValueError(f"out may hold {known} here, got {k!r}")
    for name, shape, dtype in wanted:
        t = out.get(name)
        if t is None:
            t = _empty(shape, dtype, device, stream)
        else:
            _on(t, name, dtype, shape, dev)
        r[name] = t
    return r


def _at(r, name):
    t = r.get(name)
    return None if t is None else t.data_ptr()


def linear_backward(a, w, dy, pre=None, act: str = "none", bias: bool = False, da: bool = True, dw: bool = True,
                    dw_dtype=torch.float32, out=None, workspace=None, stream=None) -> dict:
    """Gradients of linear, given dy [..., N] (bf16), the gradient of its output (and so of the residual).

    pre: what linear_train kept (not needed without an activation).  Returns a dict of da (bf16, like a), dw
    [N, K] (dw_dtype: fp32 or bf16) and, with bias, dbias (fp32 [N]); da=False / dw=False leave one out.
    Behind an activation the products take dy act'(pre) rounded to bf16.  out: None or a dict of tensors to
    write to; workspace: None or a tensor of linear_backward_workspace_bytes(M, N, K, act, bias) bytes.
    """
    dev, N, K, lead, M, lda = _product(a, w, "a", "w")
    raw = _here(dev, stream)
    shape = lead + (N,)
    ldy = _rows(dy, "dy", torch.bfloat16, shape, dev)
    code = _act_code(act)
    if code:
        if pre is None:
            raise ValueError("pre is needed behind an activation")
        _on(pre, "pre", torch.bfloat16, shape, dev)
    want = []
    if da:
        want.append(("da", a.shape, torch.bfloat16))
    if dw:
        want.append(("dw", w.shape, dw_dtype))
    if bias:
        want.append(("dbias", (N,), torch.float32))
    r = _grads(out, want, dev, a.device, stream)
    need = linear_backward_workspace_bytes(M, N, K, act, bool(bias)) if code or bias else 0
    ws = _workspace(workspace, need, dev, a, stream)
    _check(lib().diffattn_linear_backward(M, N, K, a.data_ptr(), lda, w.data_ptr(), dy.data_ptr(), ldy,
                                          pre.data_ptr() if code else None, code, _at(r, "da"), _at(r, "dw"),
                                          _dt(r["dw"]) if dw else F32, _at(r, "dbias"), _addr(ws),
                                          0 if ws is None else ws.nbytes, raw))
    return r


def _gated(x, w_gu, act, out, gu, stream):
    dev, F2, D, lead, M, ldx = _product(x, w_gu, "x", "w_gu")
    raw = _here(dev, stream)
    if F2 % 2:
        raise ValueError(f"w_gu must be [2 F, D], got {tuple(w_gu.shape)}")
    ldh = F = F2 // 2
    if out is None:
        out = _empty(lead + (F,), torch.bfloat16, x.device, stream)
    else:
        ldh = _rows(out, "out", torch.bfloat16, lead + (F,), dev)
    if gu is not None:
        _on(gu, "gu", torch.bfloat16, lead + (F2,), dev)
        gu = gu.data_ptr()
    code = ACTIVATIONS.get(act)
    if code is None:
        code = _act_code(act)
    st = lib().diffattn_gated_linear(M, D, F, x.data_ptr(), ldx, w_gu.data_ptr(), code, out.data_ptr(), ldh, gu, raw)
    if st:
        _check(st)
    return out


def gated_linear(x, w_gu, act: str = "silu", out=None, stream=None) -> torch.Tensor:
    """h = act(x Wg^T) * (x Wu^T) in one kernel: x [..., D], w_gu = [Wg; Wu] [2 F, D] (bf16) -> [..., F] bf16.

    linear(h, w_down, residual=...) is the rest of a feed-forward block.  x and out may be 2-D with rows
    further apart (multiples of 8 elements).
    """
    return _gated(x, w_gu, act, out, None, stream)


def gated_linear_train(x, w_gu, act: str = "silu", out=None, gu=None, stream=None):
    """gated_linear that also keeps [x Wg^T | x Wu^T] (bf16 [..., 2 F]) for its backward: returns (h, gu)."""
    if gu is None:
        gu = _empty(x.shape[:-1] + w_gu.shape[:1], torch.bfloat16, x.device, stream)
    return _gated(x, w_gu, act, out, gu, stream), gu


@functools.lru_cache(maxsize=1024)
def gated_linear_backward_workspace_bytes(M: int, D: int, F: int) -> int:
    return int(lib().diffattn_gated_linear_backward_workspace(M, D, F))


def gated_linear_backward(x, w_gu, gu, dh, act: str = "silu", dx: bool = True, dw: bool = True, dw_dtype=torch.float32,
                          out=None, workspace=None, stream=None) -> dict:
    """Gradients of gated_linear, given dh [..., F] (bf16) and gu as gated_linear_train kept it.

    Returns a dict of dx (bf16, like x) and dw (like w_gu, of dw_dtype: fp32 or bf16).  The products take
    the gradients of gu rounded to bf16.  out: None or a dict of tensors to write to; workspace: None or a
    tensor of gated_linear_backward_workspace_bytes(M, D, F) bytes.
    """
    dev, F2, D, lead, M, ldx = _product(x, w_gu, "x", "w_gu")
    raw = _here(dev, stream)
    if F2 % 2:
        raise ValueError(f"w_gu must be [2 F, D], got {tuple(w_gu.shape)}")
    F = F2 // 2
    _on(gu, "gu", torch.bfloat16, lead + (2 * F,), dev)
    ldh = _rows(dh, "dh", torch.bfloat16, lead + (F,), dev)
    want = []
    if dx:
        want.append(("dx", x.shape, torch.bfloat16))
    if dw:
        want.append(("dw", w_gu.shape, dw_dtype))
    r = _grads(out, want, dev, x.device, stream)
    ws = _workspace(workspace, gated_linear_backward_workspace_bytes(M, D, F), dev, x, stream)
    _check(lib().diffattn_gated_linear_backward(M, D, F, x.data_ptr(), ldx, w_gu.data_ptr(), gu.data_ptr(),
                                                dh.data_ptr(), ldh, _act_code(act), _at(r, "dx"), _at(r, "dw"),
                                                _dt(r["dw"]) if dw else F32, _addr(ws), 0 if ws is None else ws.nbytes,
                                                raw))
    return r


def _gate_rows(gate, x, dev) -> int:
    """The rows of a gate: [D], [G, D] with G dividing the rows of x, or like x."""
    if gate is None:
        return 0
    D = x.shape[-1]
    if gate.dim() == 1:
        n = 1
    elif gate.shape == x.shape:
        n = x.shape[:-1].numel()
    elif gate.dim() == 2:
        n = gate.shape[0]
        if n == 0 and x.shape[:-1].numel() > 0:
            raise ValueError(f"gate has no rows, x {tuple(x.shape)} has")
    else:
        raise ValueError(f"gate must be [D], [G, D] or like x {tuple(x.shape)}, got {tuple(gate.shape)}")
    _on(gate, "gate", torch.float32, gate.shape[:-1] + (D,), dev)
    return n


def _norm_args(x, stream_dtype, gate, gamma_post, gamma):
    """Device, width, rows, the types' codes, gate rows."""
    dev, shape, dt = x.get_device(), x.shape, x.dtype
    if dev < 0:
        raise ValueError("x must be a CUDA tensor")
    if not shape:
        raise ValueError("x must be [..., D]")
    D, rows = shape[-1], shape[:-1].numel()
    if (D | rows) >> 31:
        raise ValueError(f"x {tuple(shape)}: sizes are below 2^31")
    if not x.is_contiguous():
        _on(x, "x", dt, shape, dev)
    if gamma_post is not None:
        _on(gamma_post, "gamma_post", _f32, (D,), dev)
    if gamma is not None:
        _on(gamma, "gamma", _f32, (D,), dev)
    if stream_dtype is not _bf16 and stream_dtype is not _f32:
        raise ValueError(f"unsupported dtype {stream_dtype} (bf16 or fp32)")
    return (dev, D, rows, BF16 if dt is _bf16 else _dt(x), BF16 if stream_dtype is _bf16 else F32,
            0 if gate is None else _gate_rows(gate, x, dev))


def residual_norm(x, residual=None, gate=None, scale: float = 1.0, gamma_post=None, post=None, gamma=None,
                  norm: bool = True, eps: float = 1e-5, stream_dtype=None, out=None, y=None, stream=None):
    """The norms after and before a block with its gate and residual scale, in one pass.

    p = x / rms(x) * gamma_post (post, the default where gamma_post is given; else p = x),
    s = residual + scale * gate * p, y = s / rms(s) * gamma, over the last dimension (1 to 8192).
    x: [..., D] bf16 or fp32; residual: like x, or fp32 beside a bf16 x; gate: fp32 [D], like x, or
    [G, D] where G divides x's rows (G sequences: each its own row); gammas: fp32 [D] or None (ones).  norm=False: without the second norm.
    stream_dtype: the type of s (default the residual's or out's, else x's).  out: s, which may be residual
    itself.  eps of 0 or less selects 1e-5.  Returns (y, s); y is None without the second norm.
    """
    xdt = x.dtype
    sdt = residual.dtype if residual is not None else out.dtype if out is not None else (stream_dtype or xdt)
    if stream_dtype is not None and stream_dtype is not sdt:
        raise ValueError(f"stream_dtype is {stream_dtype}, the {'residual' if residual is not None else 'out'} given is {sdt}")
    dev, D, rows, dt, sd, gate_rows = _norm_args(x, sdt, gate, gamma_post, gamma)
    raw = _here(dev, stream)
    shape = x.shape
    if residual is not None:
        _on(residual, "residual", sdt, shape, dev)
        residual_at = residual.data_ptr()
    else:
        residual_at = None
    if out is None:
        if sdt is xdt and stream is None:
            out = torch.empty_like(x)
        else:
            out = _empty(shape, sdt, x.device, stream)
    else:
        _on(out, "out", sdt, shape, dev)
    if not norm:
        if y is not None or gamma is not None:
            raise ValueError("y and gamma belong to the second norm")
        y_at = None
    else:
        if y is None:
            y = _like(x, stream)
        else:
            _on(y, "y", xdt, shape, dev)
        y_at = y.data_ptr()
    st = lib().diffattn_residual_norm(dt, sd, rows, D, x.data_ptr(), residual_at, _addr(gate), gate_rows, scale,
                                      1 if (gamma_post is not None if post is None else post) else 0, _addr(gamma_post),
                                      _addr(gamma), eps, out.data_ptr(), y_at, raw)
    if st:
        _check(st)
    return y, out


@functools.lru_cache(maxsize=1024)
def residual_norm_backward_workspace_bytes(rows: int, D: int, gate_rows: int = 0) -> int:
    return int(lib().diffattn_residual_norm_backward_workspace(rows, D, gate_rows))


def residual_norm_backward(x, s, dy=None, ds=None, gate=None, scale: float = 1.0, gamma_post=None, post=None, gamma=None,
                           eps: float = 1e-5, out=None, workspace=None, stream=None, dx: bool = True, dresidual: bool = True,
                           dgate: bool = True, dgammas: bool = True) -> dict:
    """Gradients of residual_norm from x, the s it returned, dy (like y) and ds (like s; either may be None).

    Returns a dict of dx, dresidual (like s), and of those that apply: dgate (like gate), dgamma_post (post),
    dgamma (with dy), fp32; dx=False, dresidual=False, dgate=False and dgammas=False leave theirs out.  out:
    None or a dict of tensors to write to (dresidual may be ds); workspace: None or a tensor of
    residual_norm_backward_workspace_bytes(rows, D, gate rows) bytes.
    """
    dev, D, rows, dt, sd, gate_rows = _norm_args(x, s.dtype, gate, gamma_post, gamma)
    raw = _here(dev, stream)
    post = gamma_post is not None if post is None else bool(post)
    _on(s, "s", s.dtype, x.shape, dev)
    if dy is not None:
        _on(dy, "dy", x.dtype, x.shape, dev)
    if ds is not None:
        _on(ds, "ds", s.dtype, x.shape, dev)
    want = []
    if dx:
        want.append(("dx", x.shape, x.dtype))
    if dresidual:
        want.append(("dresidual", x.shape, s.dtype))
    if gate is not None and dgate:
        want.append(("dgate", gate.shape, torch.float32))
    if post and dgammas:
        want.append(("dgamma_post", (D,), torch.float32))
    if dy is not None and dgammas:
        want.append(("dgamma", (D,), torch.float32))
    r = _grads(out, want, dev, x.device, stream)
    ws = _workspace(workspace, residual_norm_backward_workspace_bytes(rows, D, gate_rows), dev, x, stream)
    _check(lib().diffattn_residual_norm_backward(dt, sd, rows, D, x.data_ptr(), s.data_ptr(), _addr(dy), _addr(ds),
                                                 _addr(gate), gate_rows, scale, 1 if post else 0, _addr(gamma_post),
                                                 _addr(gamma), eps, _at(r, "dx"), _at(r, "dresidual"),
                                                 _at(r, "dgate"), _at(r, "dgamma_post"), _at(r, "dgamma"),
                                                 _addr(ws), 0 if ws is None else ws.nbytes, raw))
    return r


def bounds_checked() -> bool:
    """True when the loaded library is the bounds-check build."""
    return bool(lib().diffattn_bounds_checked())


def debug_bounds_selftest(stream=None) -> None:
    """Bounds-check build: one checked store out of its limit (skipped and recorded)."""
    _check(lib().diffattn_debug_bounds_selftest(_stream(stream)))


def debug_item_plan(grid: int, units: int, nqt: int, qt0: int, n: int, causal: bool, kv_unit_bytes: int):
    """The host's item plan of a persistent d = 128 forward: (first [grid + 1], items [units nqt]) as
    numpy uint16 arrays, or None when the launch is too large for a plan."""
    import numpy as np
    first = np.zeros(max(grid, 0) + 1, dtype=np.uint16)
    items = np.zeros(max(units * nqt, 1), dtype=np.uint16)
    cnt = lib().diffattn_debug_item_plan(grid, units, nqt, qt0, n, 1 if causal else 0, kv_unit_bytes,
                                         first.ctypes.data_as(ctypes.c_void_p), items.ctypes.data_as(ctypes.c_void_p))
    return None if cnt == 0 else (first, items)


PRODUCTS = {"linear": 0, "gated": 1, "da": 2, "dw": 3}


def debug_product_plan(kind: str, M: int, N: int, K: int, f32: bool = False) -> dict:
    """How a product [M, N] over a contraction of K would run (host only).

    kind: "linear", "gated" (N = F, K = D), "da" (dx too) or "dw".  Returns a dict: kernel ("few" or "tiles") and
    its layout; segment: the values of K that one accumulator sums (f32: of an fp32 output).
    """
    plan = (ctypes.c_int * 6)()
    form = lib().diffattn_debug_product_plan(PRODUCTS[kind], M, N, K, 1 if f32 else 0, plan)
    if form == 1:
        return dict(kernel="few", cluster=plan[0], width=plan[1], tokens=plan[2], stages=plan[4], segment=plan[5])
    if form == 2:
        return dict(kernel="tiles", cluster=plan[0], whole=plan[1], halved=plan[2], segment=plan[5])
    raise ValueError(f"no product {kind} of {M} x {N} x {K}")


def device_status(stream=None) -> int:
    """Synchronise the stream, read and clear the device status word (raises on error)."""
    st = lib().diffattn_device_status(_stream(stream))
    _check(st)
    return st


def debug_wait_timeout(budget_ns: int, stream=None) -> None:
    """Launch the bounded-wait self-test kernel (its wait must run out)."""
    _check(lib().diffattn_debug_wait_timeout(int(budget_ns), _stream(stream)))


def launch_count() -> int:
    """Kernels launched by the library so far in this process."""
    return int(lib().diffattn_launch_count())
