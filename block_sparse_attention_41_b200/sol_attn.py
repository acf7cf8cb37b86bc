"""Thin ctypes binding of libsolattn.so (C ABI in include/sol_attn.h), with the same call names.

This module only marshals arguments: it checks tensor placement, dtype and contiguity,
allocates output tensors with torch when the caller passes none, passes raw pointers and
the current CUDA stream, and turns status codes into exceptions. All compute runs in the
library's CUDA kernels. There is no fallback: if the library is missing or no sm_100 GPU is
present, the calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Sequence

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsolattn.so")

SOL_OK, SOL_EINVAL, SOL_EUNSUPPORTED, SOL_ECUDA, SOL_ETIMEOUT = range(5)
SOL_F32, SOL_BF16 = 0, 1

# symbols declared in include/sol_attn.h
EXPORTED = (
    "sol_attn_status_string",
    "sol_attn_last_error",
    "sol_attn_pool",
    "sol_attn_fwd_workspace_bytes",
    "sol_attn_fwd",
    "sol_attn_check_device_error",
    "sol_attn_debug_drop_one_load",
    "sol_attn_debug_record_cta_times",
    "sol_attn_fwd_noalloc",
    "sol_attn_qknorm_rope_pool",
    "sol_attn_fwd_host_scratch_bytes",
    "sol_attn_fwd_host",
    "sol_attn_fwd_topk",
    "sol_attn_quantize_qk8",
    "sol_attn_fwd_qk8",
    "sol_attn_qknorm_rope_pool_qbar",
    "sol_attn_fwd_qbar",
    "sol_attn_quantize_v8",
    "sol_attn_fwd_8bit",
    "sol_attn_residual_norm",
    "sol_attn_residual_norm_bwd",
    "sol_attn_residual_norm_bwd_workspace_bytes",
    "sol_attn_rope_inv_freq",
    "sol_attn_rope_tables",
    "sol_attn_rope",
    "sol_attn_linear",
    "sol_attn_linear_workspace_bytes",
    "sol_attn_linear_bwd",
    "sol_attn_linear_bwd_workspace_bytes",
)

# names of the enumerations of the dense operators
NORMS = {"none": 0, "layer": 1, "rms": 2}
ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
ACTIVATIONS = {"none": 0, "gelu": 1, "gelu_tanh": 2, "silu": 3}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


class SolAttnError(RuntimeError):
    """A library call returned a status other than SOL_OK."""

    def __init__(self, status: int, call: str, detail: str):
        self.status = status
        super().__init__(f"{call}: {status_string(status)}: {detail}")


_lib = None


def load_library() -> ctypes.CDLL:
    """Load libsolattn.so once; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with `python -m block_sparse_attention_41_b200.build` "
            "(there is no non-CUDA implementation)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, f32p = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(ctypes.c_float)
    lib.sol_attn_status_string.argtypes = [i32]
    lib.sol_attn_status_string.restype = ctypes.c_char_p
    lib.sol_attn_last_error.argtypes = []
    lib.sol_attn_last_error.restype = ctypes.c_char_p
    lib.sol_attn_pool.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp]
    lib.sol_attn_pool.restype = i32
    lib.sol_attn_fwd_workspace_bytes.argtypes = [i32, i32, i32, i32]
    lib.sol_attn_fwd_workspace_bytes.restype = ctypes.c_size_t
    lib.sol_attn_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, f32p, i32, i32, i32, i32, i32, i32, i32, i32,
                                 vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.sol_attn_fwd.restype = i32
    lib.sol_attn_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, f32p, i32, i32, i32, i32, i32, i32, i32, i32,
                                         vp, vp, vp, vp]
    lib.sol_attn_fwd_noalloc.restype = i32
    lib.sol_attn_qknorm_rope_pool.argtypes = [vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, i32, i32, i32, i32, i32,
                                              vp, vp, vp, vp, vp, vp, vp]
    lib.sol_attn_qknorm_rope_pool.restype = i32
    lib.sol_attn_qknorm_rope_pool_qbar.argtypes = [vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, i32, i32, i32, i32,
                                                   i32, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.sol_attn_qknorm_rope_pool_qbar.restype = i32
    lib.sol_attn_fwd_qbar.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, f32p, i32, i32, i32, i32, i32, vp, vp, vp, vp,
                                      ctypes.c_size_t, vp]
    lib.sol_attn_fwd_qbar.restype = i32
    lib.sol_attn_quantize_v8.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, vp]
    lib.sol_attn_quantize_v8.restype = i32
    lib.sol_attn_fwd_8bit.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, f32p, i32, i32, i32, i32, i32, vp, vp,
                                      vp, vp, ctypes.c_size_t, vp]
    lib.sol_attn_fwd_8bit.restype = i32
    lib.sol_attn_quantize_qk8.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.sol_attn_quantize_qk8.restype = i32
    lib.sol_attn_fwd_qk8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, f32p, i32, i32, i32, i32, i32, vp, vp,
                                     vp, vp, ctypes.c_size_t, vp]
    lib.sol_attn_fwd_qk8.restype = i32
    lib.sol_attn_fwd_host_scratch_bytes.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    lib.sol_attn_fwd_host_scratch_bytes.restype = ctypes.c_size_t
    lib.sol_attn_fwd_host.argtypes = [vp, vp, vp, vp, f32p, i32, i32, i32, i32, i32, i32, i32, i32, vp, vp,
                                      ctypes.c_size_t, vp]
    lib.sol_attn_fwd_host.restype = i32
    lib.sol_attn_fwd_topk.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp,
                                      ctypes.c_size_t, vp]
    lib.sol_attn_fwd_topk.restype = i32
    i64, f32, f64, i64p, i32p = ctypes.c_int64, ctypes.c_float, ctypes.c_double, ctypes.POINTER(ctypes.c_int64), \
        ctypes.POINTER(ctypes.c_int)
    size = ctypes.c_size_t
    lib.sol_attn_residual_norm.argtypes = [vp, vp, vp, i64, vp, vp, i64, vp, i64, vp, i32, i32, i32, f32, f32, i32, i32,
                                           i32, vp, vp, vp]
    lib.sol_attn_residual_norm.restype = i32
    lib.sol_attn_residual_norm_bwd_workspace_bytes.argtypes = [i32, i32, i32]
    lib.sol_attn_residual_norm_bwd_workspace_bytes.restype = size
    lib.sol_attn_residual_norm_bwd.argtypes = [vp, vp, vp, vp, vp, i64, vp, vp, i64, vp, i32, i32, i32, f32, f32, i32,
                                               i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, size, vp]
    lib.sol_attn_residual_norm_bwd.restype = i32
    lib.sol_attn_rope_inv_freq.argtypes = [i32, f64, i32, i32p, i32, f64, f64, f64, f64, ctypes.POINTER(f64), f32p]
    lib.sol_attn_rope_inv_freq.restype = i32
    lib.sol_attn_rope_tables.argtypes = [vp, i32, i32p, vp, f32, i32, i32, vp, vp, vp]
    lib.sol_attn_rope_tables.restype = i32
    lib.sol_attn_rope.argtypes = [vp, i64p, vp, i64p, i32, vp, i64, i32, i32p, vp, f32, i32, i32, i32, i32, i32, i32, i32,
                                  i32, vp, i64p, vp, i64p, vp]
    lib.sol_attn_rope.restype = i32
    lib.sol_attn_linear.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, size, vp]
    lib.sol_attn_linear.restype = i32
    lib.sol_attn_linear_workspace_bytes.argtypes = [i32, i32, i32]
    lib.sol_attn_linear_workspace_bytes.restype = size
    lib.sol_attn_linear_bwd_workspace_bytes.argtypes = [i32, i32, i32]
    lib.sol_attn_linear_bwd_workspace_bytes.restype = size
    lib.sol_attn_linear_bwd.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, size, vp]
    lib.sol_attn_linear_bwd.restype = i32
    lib.sol_attn_check_device_error.argtypes = [vp, vp]
    lib.sol_attn_check_device_error.restype = i32
    lib.sol_attn_debug_drop_one_load.argtypes = [i32]
    lib.sol_attn_debug_drop_one_load.restype = None
    lib.sol_attn_debug_record_cta_times.argtypes = [vp, i32]
    lib.sol_attn_debug_record_cta_times.restype = None
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().sol_attn_status_string(int(status)).decode()


def _check(status: int, call: str) -> None:
    if status != SOL_OK:
        raise SolAttnError(status, call, load_library().sol_attn_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SOL_BF16
    if t.dtype == torch.float32:
        return SOL_F32
    raise TypeError(f"unsupported dtype {t.dtype}: use torch.bfloat16 or torch.float32")


def _need_cuda(name: str, t: torch.Tensor, dtype=None) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")


def sol_attn_pool(K: torch.Tensor, V: torch.Tensor, block_k: int, kbar=None, vbar=None, kbar_lp=None,
                  vbar_lp=None, stream=None):
    """Block means of K and V. Returns (kbar, vbar, kbar_lp, vbar_lp); the bf16 mirrors are None
    for fp32 inputs."""
    _need_cuda("K", K)
    _need_cuda("V", V, K.dtype)
    B, H, L, d = K.shape
    if V.shape != K.shape:
        raise ValueError("K and V must have the same shape")
    nkb = -(-L // block_k)
    dt = _dtype_code(K)
    dev = K.device
    if kbar is None:
        kbar = torch.empty((B, H, nkb, d), dtype=torch.float32, device=dev)
    if vbar is None:
        vbar = torch.empty((B, H, nkb, d), dtype=torch.float32, device=dev)
    if dt == SOL_BF16:
        if kbar_lp is None:
            kbar_lp = torch.empty((B, H, nkb, d), dtype=torch.bfloat16, device=dev)
        if vbar_lp is None:
            vbar_lp = torch.empty((B, H, nkb, d), dtype=torch.bfloat16, device=dev)
    for n, t in (("kbar", kbar), ("vbar", vbar)):
        _need_cuda(n, t, torch.float32)
    st = load_library().sol_attn_pool(_ptr(K), _ptr(V), dt, B, H, L, d, block_k, _ptr(kbar), _ptr(vbar),
                                      _ptr(kbar_lp), _ptr(vbar_lp), _stream(stream))
    _check(st, "sol_attn_pool")
    return kbar, vbar, kbar_lp, vbar_lp


def sol_attn_qknorm_rope_pool(Q, K, V, gain_q, gain_k, rope_cos, rope_sin, block_k: int, eps: float = 1e-6,
                              Q_out=None, K_out=None, kbar=None, vbar=None, kbar_lp=None, vbar_lp=None, stream=None,
                              qbar=None, want_qbar: bool = False):
    """QK RMS norm + rotary embedding of Q and K, and the block means of the stored K and of V, in
    one pass. Returns (Q_out, K_out, kbar, vbar, kbar_lp, vbar_lp), plus qbar (the block means of
    the stored Q, for sol_attn_fwd_qbar) when want_qbar or a qbar tensor is given. Pass Q_out=Q,
    K_out=K to work in place."""
    for n, t in (("Q", Q), ("K", K), ("V", V)):
        _need_cuda(n, t, torch.bfloat16)
    B, H, L, d = Q.shape
    if K.shape != Q.shape or V.shape != Q.shape:
        raise ValueError("Q, K and V must have the same shape [B, H, L, d]")
    for n, t in (("gain_q", gain_q), ("gain_k", gain_k), ("rope_cos", rope_cos), ("rope_sin", rope_sin)):
        _need_cuda(n, t, torch.float32)
    if rope_cos.shape != (L, d // 2) or rope_sin.shape != (L, d // 2):
        raise ValueError(f"rope tables must be [L, d/2] = [{L}, {d // 2}]")
    nkb = -(-L // block_k)
    dev = Q.device
    Q_out = torch.empty_like(Q) if Q_out is None else Q_out
    K_out = torch.empty_like(K) if K_out is None else K_out
    kbar = torch.empty((B, H, nkb, d), dtype=torch.float32, device=dev) if kbar is None else kbar
    vbar = torch.empty((B, H, nkb, d), dtype=torch.float32, device=dev) if vbar is None else vbar
    kbar_lp = torch.empty((B, H, nkb, d), dtype=torch.bfloat16, device=dev) if kbar_lp is None else kbar_lp
    vbar_lp = torch.empty((B, H, nkb, d), dtype=torch.bfloat16, device=dev) if vbar_lp is None else vbar_lp
    if qbar is None and not want_qbar:
        st = load_library().sol_attn_qknorm_rope_pool(
            _ptr(Q), _ptr(K), _ptr(V), _ptr(gain_q), _ptr(gain_k), _ptr(rope_cos), _ptr(rope_sin),
            ctypes.c_float(eps), B, H, L, d, block_k, _ptr(Q_out), _ptr(K_out), _ptr(kbar), _ptr(vbar), _ptr(kbar_lp),
            _ptr(vbar_lp), _stream(stream))
        _check(st, "sol_attn_qknorm_rope_pool")
        return Q_out, K_out, kbar, vbar, kbar_lp, vbar_lp
    qbar = torch.empty((B, H, nkb, d), dtype=torch.float32, device=dev) if qbar is None else qbar
    _need_cuda("qbar", qbar, torch.float32)
    st = load_library().sol_attn_qknorm_rope_pool_qbar(
        _ptr(Q), _ptr(K), _ptr(V), _ptr(gain_q), _ptr(gain_k), _ptr(rope_cos), _ptr(rope_sin), ctypes.c_float(eps),
        B, H, L, d, block_k, _ptr(Q_out), _ptr(K_out), _ptr(kbar), _ptr(vbar), _ptr(kbar_lp), _ptr(vbar_lp),
        _ptr(qbar), _stream(stream))
    _check(st, "sol_attn_qknorm_rope_pool_qbar")
    return Q_out, K_out, kbar, vbar, kbar_lp, vbar_lp, qbar


def sol_attn_quantize_qk8(Q, K, kbar, stream=None):
    """8-bit QK^T operands (blocks of 128): returns (q8, k8, kbar8, q_scale, k_scale, kbar_scale, mu),
    the int8 codes of Q, K - mu and kbar - mu with one scale per 128-row tile, and the mean key mu."""
    for n, t in (("Q", Q), ("K", K)):
        _need_cuda(n, t, torch.bfloat16)
    _need_cuda("kbar", kbar, torch.float32)
    B, H, L, d = Q.shape
    nkb = -(-L // 128)
    if K.shape != Q.shape or tuple(kbar.shape) != (B, H, nkb, d):
        raise ValueError("Q, K must be [B, H, L, d] and kbar [B, H, ceil(L/128), d]")
    dev = Q.device
    q8 = torch.empty((B, H, L, d), dtype=torch.int8, device=dev)
    k8 = torch.empty_like(q8)
    kbar8 = torch.empty((B, H, nkb, d), dtype=torch.int8, device=dev)
    q_scale = torch.empty((B, H, nkb), dtype=torch.float32, device=dev)
    k_scale = torch.empty_like(q_scale)
    kbar_scale = torch.empty((B, H, -(-nkb // 128)), dtype=torch.float32, device=dev)
    mu = torch.empty((B, H, d), dtype=torch.float32, device=dev)
    st = load_library().sol_attn_quantize_qk8(
        _ptr(Q), _ptr(K), _ptr(kbar), B, H, L, d, _ptr(q8), _ptr(k8), _ptr(kbar8), _ptr(q_scale), _ptr(k_scale),
        _ptr(kbar_scale), _ptr(mu), _stream(stream))
    _check(st, "sol_attn_quantize_qk8")
    return q8, k8, kbar8, q_scale, k_scale, kbar_scale, mu


def sol_attn_fwd_qk8(Q, q8, k8, kbar8, q_scale, k_scale, kbar_scale, V, kbar, vbar_lp, tau: Sequence[float],
                     n_force: int = 0, O=None, kept_mask=None, density=None, workspace=None, stream=None):
    """The forward with 8-bit QK^T from the operands of sol_attn_quantize_qk8 (d = 128). Returns O."""
    _need_cuda("Q", Q, torch.bfloat16)
    _need_cuda("V", V, torch.bfloat16)
    B, H, L, d = Q.shape
    for n, t in (("q8", q8), ("k8", k8), ("kbar8", kbar8)):
        _need_cuda(n, t, torch.int8)
    for n, t in (("q_scale", q_scale), ("k_scale", k_scale), ("kbar_scale", kbar_scale), ("kbar", kbar)):
        _need_cuda(n, t, torch.float32)
    _need_cuda("vbar_lp", vbar_lp, torch.bfloat16)
    tau = [float(x) for x in tau]
    if len(tau) != H:
        raise ValueError(f"tau must hold H={H} values")
    if O is None:
        O = torch.empty_like(Q)
    if workspace is None:
        workspace = new_workspace(B, H, L, 128, Q.device)
    tau_c = (ctypes.c_float * H)(*tau)
    st = load_library().sol_attn_fwd_qk8(
        _ptr(Q), _ptr(q8), _ptr(k8), _ptr(kbar8), _ptr(q_scale), _ptr(k_scale), _ptr(kbar_scale), _ptr(V), _ptr(kbar),
        _ptr(vbar_lp), tau_c, B, H, L, d, int(n_force), _ptr(O), _ptr(kept_mask), _ptr(density), _ptr(workspace),
        workspace.numel(), _stream(stream))
    _check(st, "sol_attn_fwd_qk8")
    return O


def sol_attn_fwd_workspace_bytes(B: int, H: int, L: int, block_q: int) -> int:
    return int(load_library().sol_attn_fwd_workspace_bytes(B, H, L, block_q))


def new_workspace(B: int, H: int, L: int, block_q: int, device) -> torch.Tensor:
    """A zeroed workspace buffer of the size sol_attn_fwd needs."""
    return torch.zeros(sol_attn_fwd_workspace_bytes(B, H, L, block_q), dtype=torch.uint8, device=device)


def sol_attn_fwd(Q, K, V, kbar, vbar, kbar_lp, vbar_lp, tau: Sequence[float], block_q: int, block_k: int,
                 n_force: int = 0, O=None, kept_mask=None, density=None, workspace=None, stream=None):
    """Fused routing + exact kept-block attention + skipped-block correction. Returns O.

    `tau` is a host sequence of H floats (>= 0, +inf = dense). `kept_mask` (uint8
    [B,H,N_qb,N_kb]) and `density` (float32 [B,H]) are optional output tensors.
    """
    _need_cuda("Q", Q)
    for n, t in (("K", K), ("V", V)):
        _need_cuda(n, t, Q.dtype)
    B, H, L, d = Q.shape
    if K.shape != Q.shape or V.shape != Q.shape:
        raise ValueError("Q, K and V must have the same shape [B, H, L, d]")
    dt = _dtype_code(Q)
    tau = [float(x) for x in tau]
    if len(tau) != H:
        raise ValueError(f"tau must hold H={H} values")
    if O is None:
        O = torch.empty_like(Q)
    if workspace is None:
        workspace = new_workspace(B, H, L, block_q, Q.device)
    tau_c = (ctypes.c_float * H)(*tau)
    st = load_library().sol_attn_fwd(
        _ptr(Q), _ptr(K), _ptr(V), _ptr(kbar), _ptr(vbar), _ptr(kbar_lp), _ptr(vbar_lp), tau_c, dt, B, H, L, d,
        block_q, block_k, int(n_force), _ptr(O), _ptr(kept_mask), _ptr(density), _ptr(workspace),
        workspace.numel(), _stream(stream))
    _check(st, "sol_attn_fwd")
    return O


def sol_attn_fwd_noalloc(Q, K, V, kbar, vbar, kbar_lp, vbar_lp, tau: Sequence[float], block_q: int, block_k: int,
                         n_force: int = 0, O=None, kept_mask=None, density=None, stream=None):
    """sol_attn_fwd without a workspace argument: the library uses its own static device array
    (B*H <= 4096; calls that overlap on the GPU race on it). For callers that cannot allocate
    device memory; pass a preallocated `O` to allocate nothing here either."""
    _need_cuda("Q", Q)
    for n, t in (("K", K), ("V", V)):
        _need_cuda(n, t, Q.dtype)
    B, H, L, d = Q.shape
    if K.shape != Q.shape or V.shape != Q.shape:
        raise ValueError("Q, K and V must have the same shape [B, H, L, d]")
    tau = [float(x) for x in tau]
    if len(tau) != H:
        raise ValueError(f"tau must hold H={H} values")
    if O is None:
        O = torch.empty_like(Q)
    tau_c = (ctypes.c_float * H)(*tau)
    st = load_library().sol_attn_fwd_noalloc(
        _ptr(Q), _ptr(K), _ptr(V), _ptr(kbar), _ptr(vbar), _ptr(kbar_lp), _ptr(vbar_lp), tau_c, _dtype_code(Q), B, H,
        L, d, block_q, block_k, int(n_force), _ptr(O), _ptr(kept_mask), _ptr(density), _stream(stream))
    _check(st, "sol_attn_fwd_noalloc")
    return O


def sol_attn_fwd_topk(Q, K, V, kbar, kbar_lp, vbar_lp, k_keep: int, n_force: int = 0, O=None, kept_mask=None,
                      density=None, workspace=None, stream=None):
    """Fused forward with fixed-sparsity routing: each query block keeps its k_keep highest-scoring
    key blocks (bf16, blocks of 128). Returns O."""
    _need_cuda("Q", Q, torch.bfloat16)
    for n, t in (("K", K), ("V", V)):
        _need_cuda(n, t, torch.bfloat16)
    B, H, L, d = Q.shape
    if K.shape != Q.shape or V.shape != Q.shape:
        raise ValueError("Q, K and V must have the same shape [B, H, L, d]")
    if O is None:
        O = torch.empty_like(Q)
    if workspace is None:
        workspace = new_workspace(B, H, L, 128, Q.device)
    st = load_library().sol_attn_fwd_topk(
        _ptr(Q), _ptr(K), _ptr(V), _ptr(kbar), _ptr(kbar_lp), _ptr(vbar_lp), int(k_keep), B, H, L, d, int(n_force),
        _ptr(O), _ptr(kept_mask), _ptr(density), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "sol_attn_fwd_topk")
    return O


def sol_attn_fwd_qbar(Q, K, V, kbar, vbar, kbar_lp, vbar_lp, qbar, tau, n_force: int = 0, O=None, kept_mask=None,
                      density=None, workspace=None, stream=None):
    """Fused forward whose routing pass takes the query-block means qbar (fp32 [B, H, N_qb, d],
    from sol_attn_qknorm_rope_pool(..., want_qbar=True)) instead of reading Q for them (bf16,
    blocks of 128). Returns O."""
    _need_cuda("Q", Q, torch.bfloat16)
    for n, t in (("K", K), ("V", V)):
        _need_cuda(n, t, torch.bfloat16)
    _need_cuda("qbar", qbar, torch.float32)
    B, H, L, d = Q.shape
    if K.shape != Q.shape or V.shape != Q.shape:
        raise ValueError("Q, K and V must have the same shape [B, H, L, d]")
    if tuple(qbar.shape) != (B, H, -(-L // 128), d):
        raise ValueError("qbar must be [B, H, ceil(L/128), d]")
    tau = [float(x) for x in tau]
    if len(tau) != H:
        raise ValueError(f"tau must hold H={H} values")
    tau_arr = (ctypes.c_float * H)(*tau)
    if O is None:
        O = torch.empty_like(Q)
    if workspace is None:
        workspace = new_workspace(B, H, L, 128, Q.device)
    st = load_library().sol_attn_fwd_qbar(
        _ptr(Q), _ptr(K), _ptr(V), _ptr(kbar), _ptr(vbar), _ptr(kbar_lp), _ptr(vbar_lp), _ptr(qbar), tau_arr, B, H, L,
        d, int(n_force), _ptr(O), _ptr(kept_mask), _ptr(density), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "sol_attn_fwd_qbar")
    return O


def sol_attn_quantize_v8(V, vbar, stream=None):
    """8-bit PV values (d = 128, blocks of 128): returns (v8t, vbar8t, v_scale), the E4M3 codes of V
    and of the pooled values vbar with one scale amax_c / 448 per channel, stored transposed
    ([B, H, d, N_kb * 128] and [B, H, d, 128 * ceil(N_kb / 128)], uint8)."""
    _need_cuda("V", V, torch.bfloat16)
    _need_cuda("vbar", vbar, torch.float32)
    B, H, L, d = V.shape
    nkb = -(-L // 128)
    if tuple(vbar.shape) != (B, H, nkb, d):
        raise ValueError("vbar must be [B, H, ceil(L/128), d]")
    dev = V.device
    v8t = torch.empty((B, H, d, nkb * 128), dtype=torch.uint8, device=dev)
    vbar8t = torch.empty((B, H, d, -(-nkb // 128) * 128), dtype=torch.uint8, device=dev)
    v_scale = torch.empty((B, H, d), dtype=torch.float32, device=dev)
    st = load_library().sol_attn_quantize_v8(_ptr(V), _ptr(vbar), B, H, L, d, _ptr(v8t), _ptr(vbar8t),
                                             _ptr(v_scale), _stream(stream))
    _check(st, "sol_attn_quantize_v8")
    return v8t, vbar8t, v_scale


def sol_attn_fwd_8bit(Q, q8, k8, kbar8, q_scale, k_scale, kbar_scale, v8t, vbar8t, v_scale, kbar, tau,
                      n_force: int = 0, O=None, kept_mask=None, density=None, workspace=None, stream=None):
    """Fused forward with 8-bit kept tiles and correction: int8 QK^T (sol_attn_quantize_qk8) and E4M3
    PV (sol_attn_quantize_v8); routing from the bf16 Q and the fp32 pooled keys. Returns O (bf16)."""
    _need_cuda("Q", Q, torch.bfloat16)
    B, H, L, d = Q.shape
    tau = [float(x) for x in tau]
    if len(tau) != H:
        raise ValueError(f"tau must hold H={H} values")
    tau_c = (ctypes.c_float * H)(*tau)
    if O is None:
        O = torch.empty_like(Q)
    if workspace is None:
        workspace = new_workspace(B, H, L, 128, Q.device)
    st = load_library().sol_attn_fwd_8bit(
        _ptr(Q), _ptr(q8), _ptr(k8), _ptr(kbar8), _ptr(q_scale), _ptr(k_scale), _ptr(kbar_scale), _ptr(v8t),
        _ptr(vbar8t), _ptr(v_scale), _ptr(kbar), tau_c, B, H, L, d, int(n_force), _ptr(O), _ptr(kept_mask),
        _ptr(density), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "sol_attn_fwd_8bit")
    return O


def sol_attn_check_device_error(workspace: torch.Tensor, stream=None) -> None:
    """Synchronise and raise SolAttnError(SOL_ETIMEOUT) if a bounded device wait expired."""
    _check(load_library().sol_attn_check_device_error(_ptr(workspace), _stream(stream)),
           "sol_attn_check_device_error")


def sol_attn_debug_drop_one_load(mode: int) -> None:
    load_library().sol_attn_debug_drop_one_load(int(mode))


def sol_attn_debug_record_cta_times(times: torch.Tensor, capacity: int) -> None:
    """Arm the next bf16 fused launch to write each CTA's (start, finish) globaltimer stamps into
    `times` (int64 device tensor of at least 2 * capacity elements)."""
    _need_cuda("times", times, torch.int64)
    if times.numel() < 2 * capacity:
        raise ValueError("times must hold 2 * capacity values")
    load_library().sol_attn_debug_record_cta_times(_ptr(times), int(capacity))


def sol_attn(Q, K, V, tau, block: int = 128, n_force: int = 0, want_mask: bool = False,
             want_density: bool = False, workspace=None, stream=None):
    """The whole path for one call: pool K/V, then the fused forward.

    Returns (O, kept_mask or None, density or None).
    """
    B, H, L, d = Q.shape
    kbar, vbar, kbar_lp, vbar_lp = sol_attn_pool(K, V, block, stream=stream)
    nb = -(-L // block)
    mask = torch.empty((B, H, nb, nb), dtype=torch.uint8, device=Q.device) if want_mask else None
    dens = torch.empty((B, H), dtype=torch.float32, device=Q.device) if want_density else None
    O = sol_attn_fwd(Q, K, V, kbar, vbar, kbar_lp, vbar_lp, tau, block, block, n_force, kept_mask=mask,
                     density=dens, workspace=workspace, stream=stream)
    return O, mask, dens


def sol_attn_fwd_host_scratch_bytes(dtype: torch.dtype, B: int, H: int, L: int, d: int, block: int,
                                    heads_per_chunk: int) -> int:
    code = SOL_BF16 if dtype == torch.bfloat16 else SOL_F32 if dtype == torch.float32 else -1
    return int(load_library().sol_attn_fwd_host_scratch_bytes(code, B, H, L, d, block, heads_per_chunk))


def default_heads_per_chunk(H: int) -> int:
    """About 20 chunks per batch entry: the pipeline fills after one small upload."""
    return max(1, -(-H // 20))


def sol_attn_fwd_host(Q, K, V, tau, block: int = 128, n_force: int = 0, heads_per_chunk: Optional[int] = None,
                      O=None, want_density: bool = False, scratch=None, stream=None):
    """The whole path (pool + forward) on HOST tensors, pipelined by head chunks through device
    scratch. Synchronous: returns (O, density or None) with both in host memory.

    Q, K, V: CPU tensors [B, H, L, d] (pinned for copy/compute overlap). `scratch`: a CUDA uint8
    tensor of at least sol_attn_fwd_host_scratch_bytes(...) bytes on the current device.
    """
    for n, t in (("Q", Q), ("K", K), ("V", V)):
        if not isinstance(t, torch.Tensor) or t.device.type != "cpu":
            raise TypeError(f"{n} must be a CPU tensor")
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
        if t.dtype != Q.dtype or t.shape != Q.shape:
            raise ValueError("Q, K and V must have the same dtype and shape [B, H, L, d]")
    B, H, L, d = Q.shape
    dt = _dtype_code(Q)
    tau = [float(x) for x in tau]
    if len(tau) != H:
        raise ValueError(f"tau must hold H={H} values")
    c = default_heads_per_chunk(H) if heads_per_chunk is None else int(heads_per_chunk)
    pinned = Q.is_pinned()
    if O is None:
        O = torch.empty(Q.shape, dtype=Q.dtype, pin_memory=pinned)
    elif O.device.type != "cpu" or not O.is_contiguous() or O.dtype != Q.dtype or O.shape != Q.shape:
        raise ValueError("O must be a contiguous CPU tensor of Q's dtype and shape")
    dens = torch.empty((B, H), dtype=torch.float32, pin_memory=pinned) if want_density else None
    if scratch is None:
        scratch = torch.empty(sol_attn_fwd_host_scratch_bytes(Q.dtype, B, H, L, d, block, c), dtype=torch.uint8,
                              device=torch.device("cuda", torch.cuda.current_device()))
    else:
        _need_cuda("scratch", scratch, torch.uint8)
    tau_c = (ctypes.c_float * H)(*tau)
    st = load_library().sol_attn_fwd_host(
        _ptr(Q), _ptr(K), _ptr(V), _ptr(O), tau_c, dt, B, H, L, d, block, int(n_force), c, _ptr(dens),
        _ptr(scratch), scratch.numel(), _stream(stream))
    _check(st, "sol_attn_fwd_host")
    return O, dens


def tau_list(values) -> list:
    """Turn a JSON-style tau list ("inf" strings allowed) into floats."""
    return [math.inf if (isinstance(v, str) and v.lower() == "inf") else float(v) for v in values]


# ---- dense operators around the attention ----------------------------------------------------------

# These calls can be as short as a few microseconds on the device, so what the host does per call counts:
# addresses go to ctypes as plain integers, the stream comes as its raw handle, outputs are made by an
# input's new_empty or empty_like, and each tensor is asked one whole question (_fits) before the checks
# that find out what is wrong with it. Together they took a call on four tokens from 22 to 15 us.
_I64x3 = ctypes.c_int64 * 3
_F32, _BF16 = torch.float32, torch.bfloat16
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # torch built without CUDA has no tensors for these calls


def _fits(t, index: int, dtype, shape) -> bool:
    """A contiguous tensor on CUDA device `index` of the given dtype and shape?"""
    try:
        return t.get_device() == index and t.dtype is dtype and t.shape == shape and t.is_contiguous()
    except (AttributeError, RuntimeError):
        return False


def _elsewhere(x, stream) -> bool:
    """Does a call on x have to change the current device or stream first?"""
    return stream is not None or torch.cuda.current_device() != x.get_device()


def _addr(t):
    return None if t is None else t.data_ptr()


class _On:
    """The tensors' device made current, and the caller's stream (default: the device's current one)
    made torch's, so that what a call allocates belongs to the stream that its kernels run on."""

    __slots__ = ("device", "stream", "_contexts")

    def __init__(self, device, stream):
        self.device, self.stream, self._contexts = device, stream, ()

    def __enter__(self):
        index = self.device.index
        if self.stream is not None:
            s = self.stream
            if not hasattr(s, "cuda_stream"):  # a handle; torch takes 0, the default stream's, for a wish for a new stream
                s = torch.cuda.ExternalStream(int(s), device=self.device) if int(s) else torch.cuda.default_stream(self.device)
            elif s.device != self.device:
                raise ValueError(f"the stream is on {s.device}, the tensors on {self.device}")
            self._contexts = (torch.cuda.stream(s),)
        elif torch.cuda.current_device() != index:
            self._contexts = (torch.cuda.device(self.device),)
        for c in self._contexts:
            c.__enter__()

    def __exit__(self, *exc):
        for c in self._contexts:
            c.__exit__(*exc)
        return False


def _need_cuda_on(name: str, t, device, dtype=None) -> None:
    """_need_cuda without the contiguity, on the given device."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")


def _need_like(name: str, t, ref) -> None:
    """A contiguous CUDA tensor of ref's device, dtype and shape."""
    if _fits(t, ref.get_device(), ref.dtype, ref.shape):
        return
    _need_cuda_on(name, t, ref.device, ref.dtype)
    if t.shape != ref.shape:
        raise ValueError(f"{name} must have shape {tuple(ref.shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_vector(name: str, t, device, C: int) -> None:
    if t is None or _fits(t, device.index, _F32, (C,)):
        return
    _need_cuda_on(name, t, device, torch.float32)
    if t.shape != (C,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {C} values")


def _need_rows(name: str, t, device, B: int, C: int) -> int:
    """Checks [B, C] fp32 rows (channels contiguous) and returns their stride."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.get_device() != device.index or t.dtype is not _F32:
        _need_cuda_on(name, t, device, _F32)
    if t.shape != (B, C):
        raise ValueError(f"{name} must be [B, C] = [{B}, {C}], got {tuple(t.shape)}")
    row, channel = t.stride()
    if C > 1 and channel != 1:
        raise ValueError(f"{name}'s channels must be contiguous")
    return row if B > 1 else 0


def _choice(name: str, value, names: dict) -> int:
    try:
        return names[value]
    except (KeyError, TypeError):  # TypeError: not hashable
        raise ValueError(f"{name} must be one of {sorted(names)}, got {value!r}") from None


def _check_norm(x, y, gate, gain, scale, shift, post_gain):
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("x must be a CUDA tensor")
    if x.dim() != 3 or not x.is_contiguous():
        raise ValueError("x must be a contiguous [B, T, C] tensor")
    B, T, C = x.shape
    if y is not None:
        _need_like("y", y, x)
    _need_vector("gain", gain, x.device, C)
    _need_vector("post_gain", post_gain, x.device, C)
    dev = x.device
    return (B, T, C, _need_rows("gate", gate, dev, B, C), _need_rows("scale", scale, dev, B, C),
            _need_rows("shift", shift, dev, B, C))


def sol_attn_residual_norm(x, y=None, gate=None, gain=None, scale=None, shift=None, post_gain=None, norm="layer",
                           post_norm="none", res_scale: float = 1.0, eps: float = 1e-6, x_out=None, h=None, stream=None):
    """x' = res_scale x + gate * post_norm(y) post_gain and h = norm(x') gain (1 + scale) + shift, in one
    pass. x, y: [B, T, C]; gate, scale, shift: fp32 [B, C] (row stride free); gain, post_gain: fp32
    [C]; norms "layer" or "rms", post_norm also "none". Returns (x', h); without y, (x, h)."""
    B, T, C, gs, ss, hs = _check_norm(x, y, gate, gain, scale, shift, post_gain)
    dt, n, pn = _dtype_code(x), _choice("norm", norm, NORMS), _choice("post_norm", post_norm, NORMS)
    if x_out is not None:
        _need_like("x_out", x_out, x)
    if h is not None:
        _need_like("h", h, x)
    if _elsewhere(x, stream):
        with _On(x.device, stream):
            return sol_attn_residual_norm(x, y, gate, gain, scale, shift, post_gain, norm, post_norm, res_scale, eps, x_out, h)
    if y is not None and x_out is None:
        x_out = torch.empty_like(x)
    if h is None:
        h = torch.empty_like(x)
    st = load_library().sol_attn_residual_norm(
        x.data_ptr(), None if y is None else y.data_ptr(), None if gate is None else gate.data_ptr(), gs,
        None if gain is None else gain.data_ptr(), None if scale is None else scale.data_ptr(), ss,
        None if shift is None else shift.data_ptr(), hs, None if post_gain is None else post_gain.data_ptr(), dt, n, pn,
        res_scale, eps, B, T, C, None if x_out is None else x_out.data_ptr(), h.data_ptr(), _raw_stream(x.get_device()))
    if st != SOL_OK:
        _check(st, "sol_attn_residual_norm")
    return (x if y is None else x_out), h


def sol_attn_residual_norm_bwd(dh, x, y=None, gate=None, gain=None, scale=None, post_gain=None, dx_out=None,
                               norm="layer", post_norm="none", res_scale: float = 1.0, eps: float = 1e-6,
                               want_dshift: Optional[bool] = None, workspace=None, stream=None) -> dict:
    """Gradients of sol_attn_residual_norm from its inputs, dh (gradient of h) and dx_out (what reaches
    x' from elsewhere). Returns a dict of dx, dy and, for each vector given, dgate, dgain, dscale,
    dpost_gain (fp32, the vector's shape), and dshift where want_dshift (default: with scale); None
    for the others."""
    B, T, C, gs, ss, _ = _check_norm(x, y, gate, gain, scale, None, post_gain)
    dt, n, pn = _dtype_code(x), _choice("norm", norm, NORMS), _choice("post_norm", post_norm, NORMS)
    _need_like("dh", dh, x)
    if dx_out is not None:
        _need_like("dx_out", dx_out, x)
    _error_words(workspace, x.device)
    want_dshift = scale is not None if want_dshift is None else want_dshift
    if _elsewhere(x, stream):
        with _On(x.device, stream):
            return sol_attn_residual_norm_bwd(dh, x, y, gate, gain, scale, post_gain, dx_out, norm, post_norm, res_scale, eps,
                                              want_dshift, workspace)
    lib = load_library()

    def new(want, *shape):
        return x.new_empty(shape, dtype=_F32) if want else None
    g = {"dx": torch.empty_like(x), "dy": None if y is None else torch.empty_like(x),
         "dgate": new(gate is not None, B, C), "dgain": new(gain is not None, C),
         "dscale": new(scale is not None, B, C), "dshift": new(want_dshift, B, C),
         "dpost_gain": new(post_gain is not None, C)}
    if workspace is None and (gate is not None or gain is not None or scale is not None or want_dshift or post_gain is not None):
        workspace = x.new_empty(lib.sol_attn_residual_norm_bwd_workspace_bytes(B, T, C), dtype=torch.uint8)
    a = [None if t is None else t.data_ptr() for t in (dh, dx_out, x, y, gate, gain, scale, post_gain, *g.values(), workspace)]
    st = lib.sol_attn_residual_norm_bwd(*a[:5], gs, *a[5:7], ss, a[7], dt, n, pn, res_scale, eps, B, T, C, *a[8:],
                                        0 if workspace is None else workspace.numel(), _raw_stream(x.get_device()))
    if st != SOL_OK:
        _check(st, "sol_attn_residual_norm_bwd")
    return g


def _int_array(values):
    return None if values is None else (ctypes.c_int * len(values))(*[int(v) for v in values])


def sol_attn_rope_inv_freq(rot: int, base: float = 10000.0, sections=None, scaling: str = "none", factor: float = 1.0,
                           original_length: float = 8192.0, turns_low: float = 1.0, turns_high: float = 32.0,
                           device=None):
    """Angular step of each rotary pair (float64 [rot / 2], on `device`, default CPU) and the factor on
    cosine and sine. sections: pairs per position axis (default: one axis)."""
    n = len(sections) if sections is not None else 1
    f = torch.empty(max(int(rot) // 2, 1), dtype=torch.float64)
    m = ctypes.c_float(1.0)
    st = load_library().sol_attn_rope_inv_freq(
        int(rot), base, n, _int_array(sections), _choice("scaling", scaling, ROPE_SCALINGS), factor, original_length,
        turns_low, turns_high, ctypes.cast(ctypes.c_void_p(f.data_ptr()), ctypes.POINTER(ctypes.c_double)),
        ctypes.byref(m))
    _check(st, "sol_attn_rope_inv_freq")
    return (f if device is None else f.to(device)), float(m.value)


def _check_positions(pos, inv_freq, sections, device, L: int, B: Optional[int]):
    """(axes, sections array, stride of a batch entry's positions)."""
    axes = len(sections) if sections is not None else 1
    if not (_fits(pos, device.index, torch.int32, (axes, L)) and isinstance(inv_freq, torch.Tensor) and
            inv_freq.get_device() == device.index and inv_freq.dtype is torch.float64 and inv_freq.dim() == 1 and
            inv_freq.is_contiguous()):
        _need_cuda_on("pos", pos, device, torch.int32)
        _need_cuda_on("inv_freq", inv_freq, device, torch.float64)
        if not pos.is_contiguous() or not inv_freq.is_contiguous() or inv_freq.dim() != 1:
            raise ValueError("pos and inv_freq must be contiguous, inv_freq a vector")
        shapes = [(axes, L)] + ([(L,)] if axes == 1 else []) + ([(B, axes, L)] if B is not None else [])
        if tuple(pos.shape) not in shapes:
            raise ValueError(f"pos must have one of the shapes {shapes}, got {tuple(pos.shape)}")
    return axes, _int_array(sections), (axes * L if pos.dim() == 3 else 0)


def sol_attn_rope_tables(pos, inv_freq, sections=None, attn_factor: float = 1.0, rope_cos=None, rope_sin=None,
                         stream=None):
    """Cosine and sine tables (fp32 [L, rot / 2]) for sol_attn_qknorm_rope_pool: pos int32 [L] or
    [axes, L], inv_freq float64 [rot / 2]. Returns (rope_cos, rope_sin)."""
    if not isinstance(pos, torch.Tensor) or not pos.is_cuda:
        raise TypeError("pos must be a CUDA tensor")
    dev, L = pos.device, pos.shape[-1] if pos.dim() else 0
    axes, sec, _ = _check_positions(pos, inv_freq, sections, dev, L, None)
    half = inv_freq.numel()
    for n, t in (("rope_cos", rope_cos), ("rope_sin", rope_sin)):
        if t is not None:
            _need_cuda_on(n, t, dev, torch.float32)
            if tuple(t.shape) != (L, half) or not t.is_contiguous():
                raise ValueError(f"{n} must be a contiguous [{L}, {half}] tensor")
    if _elsewhere(pos, stream):
        with _On(dev, stream):
            return sol_attn_rope_tables(pos, inv_freq, sections, attn_factor, rope_cos, rope_sin)
    rope_cos = pos.new_empty((L, half), dtype=_F32) if rope_cos is None else rope_cos
    rope_sin = pos.new_empty((L, half), dtype=_F32) if rope_sin is None else rope_sin
    st = load_library().sol_attn_rope_tables(pos.data_ptr(), axes, sec, inv_freq.data_ptr(), attn_factor, L, 2 * half,
                                             rope_cos.data_ptr(), rope_sin.data_ptr(), _raw_stream(pos.get_device()))
    if st != SOL_OK:
        _check(st, "sol_attn_rope_tables")
    return rope_cos, rope_sin


def sol_attn_rope(Q, K, pos, inv_freq, layout: str = "interleaved", sections=None, attn_factor: float = 1.0,
                  inverse: bool = False, Q_out=None, K_out=None, stream=None):
    """Rotary positions of Q [B, Hq, L, d] and K [B, Hk, L, d] (or None), any strides with contiguous
    channels; pos int32 [L], [axes, L] or [B, axes, L]; inv_freq float64 [rot / 2] from
    sol_attn_rope_inv_freq. inverse=True turns back: the gradient. Outputs default to contiguous
    tensors; pass Q_out=Q, K_out=K to work in place. Returns (Q_out, K_out)."""
    if not isinstance(Q, torch.Tensor) or not Q.is_cuda:
        raise TypeError("Q must be a CUDA tensor")
    if Q.dim() != 4:
        raise ValueError("Q must be [B, Hq, L, d]")
    B, Hq, L, d = Q.shape
    dt, lay = _dtype_code(Q), _choice("layout", layout, ROPE_LAYOUTS)
    index, dtype = Q.get_device(), Q.dtype
    if K is None:
        if K_out is not None:
            raise ValueError("K_out needs K")
    else:
        if not isinstance(K, torch.Tensor) or K.get_device() != index or K.dtype is not dtype:
            _need_cuda_on("K", K, Q.device, dtype)
        if K.dim() != 4 or K.shape[0] != B or K.shape[2] != L or K.shape[3] != d:
            raise ValueError("K must be [B, Hk, L, d] with the B, L and d of Q")
    for n, t, ref in (("Q_out", Q_out, Q), ("K_out", K_out, K)):
        if t is not None:
            _need_cuda_on(n, t, Q.device, dtype)
            if t.shape != ref.shape:
                raise ValueError(f"{n} must have shape {tuple(ref.shape)}")
    axes, sec, pos_b = _check_positions(pos, inv_freq, sections, Q.device, L, B)
    if _elsewhere(Q, stream):
        with _On(Q.device, stream):
            return sol_attn_rope(Q, K, pos, inv_freq, layout, sections, attn_factor, inverse, Q_out, K_out)
    if Q_out is None:
        Q_out = torch.empty_like(Q, memory_format=torch.contiguous_format)
    if K is not None and K_out is None:
        K_out = torch.empty_like(K, memory_format=torch.contiguous_format)

    def rows(name, t):
        if t is None:
            return None, None
        b, h, l, c = t.stride()
        if d > 1 and c != 1:
            raise ValueError(f"{name}'s channels must be contiguous")
        return t.data_ptr(), _I64x3(b, h, l)
    st = load_library().sol_attn_rope(
        *rows("Q", Q), *rows("K", K), dt, pos.data_ptr(), pos_b, axes, sec, inv_freq.data_ptr(), attn_factor, lay,
        1 if inverse else 0, B, Hq, 0 if K is None else K.shape[1], L, d, 2 * inv_freq.numel(), *rows("Q_out", Q_out),
        *rows("K_out", K_out), _raw_stream(index))
    if st != SOL_OK:
        _check(st, "sol_attn_rope")
    return Q_out, K_out


def _check_linear(**operands):
    """A product's bf16 operands by name, w among them: contiguous, on the device of the first."""
    a = next(iter(operands.values()))
    if not isinstance(a, torch.Tensor) or not a.is_cuda:
        raise TypeError(f"{next(iter(operands))} must be a CUDA tensor")
    index = a.get_device()
    for n, t in operands.items():
        if not isinstance(t, torch.Tensor) or t.get_device() != index or t.dtype is not _BF16:
            _need_cuda_on(n, t, a.device, _BF16)
        if not t.is_contiguous() or t.dim() < 1:
            raise ValueError(f"{n} must be contiguous")
    if operands["w"].dim() != 2:
        raise ValueError("w must be [N, K]")


def _error_words(workspace, device):
    if workspace is not None:
        _need_cuda_on("workspace", workspace, device, torch.uint8)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")


def sol_attn_linear(x, w, bias=None, act: str = "none", residual=None, out=None, z=None, want_z: bool = False,
                    workspace=None, stream=None):
    """residual + act(x w^T + bias): x bf16 [..., K], w bf16 [N, K], bias fp32 [N], residual bf16 [..., N];
    act "none", "gelu", "gelu_tanh" or "silu". Returns out, or (out, z) with z = x w^T + bias (bf16, for
    sol_attn_linear_bwd) when want_z or a z tensor is given. workspace: a uint8 tensor whose first 256 bytes
    are zeroed, for sol_attn_check_device_error; with sol_attn_linear_workspace_bytes bytes (the default)
    a product of few tiles is split along K."""
    _check_linear(x=x, w=w)
    code = _choice("act", act, ACTIVATIONS)
    N, K = w.shape
    if x.shape[-1] != K:
        raise ValueError(f"x must be [..., K] with w's K = {K}, got {tuple(x.shape)}")
    shape = x.shape[:-1] + (N,)
    M = 1
    for n in x.shape[:-1]:
        M *= n
    _need_vector("bias", bias, x.device, N)
    index = x.get_device()
    for n, t in (("residual", residual), ("out", out), ("z", z)):
        if t is not None and not _fits(t, index, _BF16, shape):
            _need_cuda_on(n, t, x.device, _BF16)
            raise ValueError(f"{n} must be contiguous with shape {tuple(shape)}")
    _error_words(workspace, x.device)
    if _elsewhere(x, stream):
        with _On(x.device, stream):
            return sol_attn_linear(x, w, bias, act, residual, out, z, want_z, workspace)
    lib = load_library()
    if out is None:
        out = x.new_empty(shape)
    if z is None and want_z:
        z = x.new_empty(shape)
    if workspace is None and M > 128:
        n = lib.sol_attn_linear_workspace_bytes(M, N, K)
        if n > 256:  # the product wants to be split
            workspace = x.new_empty(n, dtype=torch.uint8)
    st = lib.sol_attn_linear(
        x.data_ptr(), w.data_ptr(), None if bias is None else bias.data_ptr(),
        None if residual is None else residual.data_ptr(), code, M, N, K, out.data_ptr(), None if z is None else z.data_ptr(),
        None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel(), _raw_stream(index))
    if st != SOL_OK:
        _check(st, "sol_attn_linear")
    return out if z is None else (out, z)


def sol_attn_linear_bwd(dy, x, w, z=None, act: str = "none", want_dx: bool = True, want_dw: bool = True,
                        want_db: bool = True, workspace=None, stream=None):
    """Gradients of sol_attn_linear from dy bf16 [..., N], its inputs and, with an activation, the z that it
    returned. Returns (dx, dw, db), bf16, bf16 and fp32, None where not wanted; residual's is dy."""
    _check_linear(dy=dy, w=w, x=x)
    code = _choice("act", act, ACTIVATIONS)
    N, K = w.shape
    if dy.shape[-1] != N or x.shape != dy.shape[:-1] + (K,):
        raise ValueError(f"dy must be [..., {N}] and x [..., {K}] with the same rows, got {tuple(dy.shape)} and {tuple(x.shape)}")
    M = 1
    for n in dy.shape[:-1]:
        M *= n
    if z is not None:
        _need_like("z", z, dy)
    _error_words(workspace, dy.device)
    if _elsewhere(dy, stream):
        with _On(dy.device, stream):
            return sol_attn_linear_bwd(dy, x, w, z, act, want_dx, want_dw, want_db, workspace)
    lib = load_library()
    dx = torch.empty_like(x) if want_dx else None
    dw = torch.empty_like(w) if want_dw else None
    db = dy.new_empty(N, dtype=_F32) if want_db else None
    if workspace is None:
        workspace = dy.new_empty(lib.sol_attn_linear_bwd_workspace_bytes(M, N, code), dtype=torch.uint8)
    st = lib.sol_attn_linear_bwd(_addr(dy), _addr(x), _addr(w), _addr(z), code, M, N, K, _addr(dx), _addr(dw), _addr(db),
                                 _addr(workspace), workspace.numel(), _raw_stream(dy.get_device()))
    if st != SOL_OK:
        _check(st, "sol_attn_linear_bwd")
    return dx, dw, db
