"""ctypes binding of ``libliger_attn.so`` (C ABI in ``include/liger_attn.h``).

Argument marshalling only: every step of the forward pass runs in the CUDA
library.  PyTorch supplies device memory and streams.  The library is loaded
on first use; if it is missing this raises (there is no CPU fallback).
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libliger_attn.so")

LIGER_OK, LIGER_ERR_INVALID_ARG, LIGER_ERR_UNSUPPORTED, LIGER_ERR_CUDA, LIGER_ERR_TIMEOUT = range(5)
LIGER_BF16, LIGER_FP32 = 0, 1
LIGER_KV_E4M3, LIGER_KV_INT8 = 0, 1
KV_CACHE_MAX_NEW = 16        # new tokens a sequence that cached_attention takes
STATUS_NAMES = {0: "LIGER_OK", 1: "LIGER_ERR_INVALID_ARG", 2: "LIGER_ERR_UNSUPPORTED",
                3: "LIGER_ERR_CUDA", 4: "LIGER_ERR_TIMEOUT"}

_vp = ctypes.c_void_p
_i = ctypes.c_int
_lock = threading.Lock()
_lib = None

# Entry points and their C signatures (restype, argtypes), as declared in the header.
SIGNATURES = {
    "liger_abi_version": (_i, []),
    "liger_last_error": (ctypes.c_char_p, []),
    "liger_attn_prefill_workspace_size": (ctypes.c_size_t, [_i, _i, _i, _i, _i, _i, _i]),
    "liger_attn_prefill": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, ctypes.c_float, _i,
                                _vp, _vp, _i, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "liger_attn_decode": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, ctypes.c_float,
                               _i, _vp]),
    "liger_attn_decode_kvshared": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, ctypes.c_float,
                                        _i, _vp]),
    "liger_attn_prefill_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, ctypes.c_float,
                                        _i, _vp, _vp, _i, _vp, _vp, _vp]),
    "liger_attn_prefill_status": (_i, [_vp, ctypes.c_size_t]),
    "liger_attn_prefill_noalloc_status": (_i, []),
    "liger_attn_prefill_plan": (_i, [_i, _i, _i, _i, _i, _i, _i, ctypes.POINTER(_i), ctypes.POINTER(_i),
                                     ctypes.POINTER(_i), ctypes.POINTER(_i), ctypes.POINTER(ctypes.c_size_t)]),
    "liger_attn_prefill_backward_workspace_size": (ctypes.c_size_t, [_i, _i, _i, _i, _i, _i, _i]),
    "liger_attn_prefill_backward": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, ctypes.c_float, _i,
                                         _vp, _i, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "liger_attn_prefill_vector_gate_workspace_size": (ctypes.c_size_t, [_i, _i, _i, _i, _i, _i, _i]),
    "liger_attn_prefill_vector_gate": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, ctypes.c_float,
                                            _i, _vp, _vp, _i, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "liger_attn_decode_vector_gate": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, ctypes.c_float,
                                           _i, _vp]),
    "liger_attn_full_causal": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _i, _i, _vp]),
    "liger_attn_full_causal_status": (_i, []),
    "liger_attn_decode_status": (_i, []),
    "liger_kv_cache_assign": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]),
    "liger_kv_cache_append": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, ctypes.c_longlong, ctypes.c_longlong,
                                   _i, _i, _vp]),
    "liger_attn_cached_workspace_size": (ctypes.c_size_t, [_i]),
    "liger_attn_cached": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, ctypes.c_longlong, _i, _i,
                               _vp, ctypes.c_size_t, _vp]),
    "liger_attn_cached_status": (_i, []),
    "liger_set_timing_events": (None, [_vp, _vp]),
    "liger_kernel_launches": (ctypes.c_uint64, []),
}


class LigerError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def load(path: Optional[str] = None):
    """Load the CUDA library (raises FileNotFoundError if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            p = path or LIB_PATH
            if not os.path.exists(p):
                raise FileNotFoundError(
                    f"{p} is missing: build it with `python -m gated_linear_attention_liger_b200.build`"
                    " (the Liger Attention ops have no CPU fallback)")
            lib = ctypes.CDLL(p)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def set_timing_events(start=None, stop=None):
    """Bracket the dominant kernel of later calls (this thread) with two torch.cuda.Events."""
    load().liger_set_timing_events(None if start is None else ctypes.c_void_p(start.cuda_event),
                                   None if stop is None else ctypes.c_void_p(stop.cuda_event))


def kernel_launches() -> int:
    """Kernels this thread has launched through the library so far."""
    return int(load().liger_kernel_launches())


def last_error() -> str:
    return load().liger_last_error().decode()


def _check(status: int):
    if status != LIGER_OK:
        raise LigerError(status, last_error())


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return LIGER_BF16
    if t.dtype == torch.float32:
        return LIGER_FP32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need_cuda(*ts):
    ref = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")
        if ref is None:
            ref = t.device
        elif t.device != ref:
            raise ValueError(f"tensors must be on one device ({ref} and {t.device})")


def _expect(t, name, shape, dtype):
    """The library sees only pointers: shapes and dtypes are checked here, so that a wrong
    output buffer is an error instead of an out-of-bounds write."""
    if t is None:
        return
    if t.shape != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def prefill_workspace_size(B, Hq, Hkv, T, d, n_seqs, dtype=torch.bfloat16) -> int:
    return int(load().liger_attn_prefill_workspace_size(
        B, Hq, Hkv, T, d, n_seqs, LIGER_BF16 if dtype == torch.bfloat16 else LIGER_FP32))


def prefill_plan(B, Hq, Hkv, T, d, n_seqs=None, packed: bool = False) -> dict:
    """The tensor-core prefill's launch plan for these sizes (host only; see the header)."""
    lib = load()
    vals = [_i(), _i(), _i(), _i()]
    nbytes = ctypes.c_size_t()
    n = B if n_seqs is None else n_seqs
    st = lib.liger_attn_prefill_plan(B, Hq, Hkv, T, d, n, int(bool(packed)), *(ctypes.byref(x) for x in vals),
                                     ctypes.byref(nbytes))
    _check(st)
    return {"chunks_per_segment": vals[0].value, "max_segments": vals[1].value,
            "state_subsegments": vals[2].value, "sm_count": vals[3].value, "plan_bytes": nbytes.value}


def prefill(q, k, v, alpha: float = 0.5, w: int = 64, initial_state=None, cu_seqlens=None,
            return_ring: bool = False, out=None, final_state=None, ring=None, pos=None,
            workspace=None, want_final_state: bool = True, stream=None):
    """Liger Attention prefill.

    q [B, T, Hq, d], k and v [B, T, Hkv, d] (bf16 or fp32, CUDA).  Returns
    (out, final_state) or, with return_ring, (out, final_state, ring, pos).
    cu_seqlens: int32 CUDA tensor of n+1 offsets (B must be 1).
    """
    lib = load()
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B, T, Hq, d] and k, v [B, T, Hkv, d]")
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    _expect(k, "k", (B, T, Hkv, d), q.dtype)
    _expect(v, "v", (B, T, Hkv, d), q.dtype)
    if cu_seqlens is not None and (cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2
                                   or cu_seqlens.dtype != torch.int32):
        raise ValueError("cu_seqlens must be a 1-D int32 tensor of n + 1 offsets")
    n = B if cu_seqlens is None else cu_seqlens.numel() - 1
    _expect(initial_state, "initial_state", (n, Hq, d, d), torch.float32)
    _expect(out, "out", (B, T, Hq, d), q.dtype)
    _expect(final_state, "final_state", (n, Hq, d, d), torch.float32)
    _expect(ring, "ring", (n, Hkv, 2, w, d), q.dtype)
    _expect(pos, "pos", (n,), torch.int32)
    _need_cuda(q, k, v, initial_state, cu_seqlens, out, final_state, ring, pos, workspace)
    dev = q.device
    if out is None:
        out = torch.empty_like(q)
    if final_state is None and want_final_state:
        final_state = torch.empty(n, Hq, d, d, device=dev, dtype=torch.float32)
    if return_ring:
        if ring is None:
            ring = torch.empty(n, Hkv, 2, w, d, device=dev, dtype=q.dtype)
        if pos is None:
            pos = torch.empty(n, device=dev, dtype=torch.int32)
    need = prefill_workspace_size(B, Hq, Hkv, T, d, n, q.dtype)
    if workspace is None and need:
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.liger_attn_prefill(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(final_state), B, Hq, Hkv, T, d, w,
        float(alpha), _dt(q), _ptr(initial_state), _ptr(cu_seqlens), n, _ptr(ring), _ptr(pos),
        _ptr(workspace), ws_bytes, _stream_ptr(stream))
    _check(st)
    if return_ring:
        return out, final_state, ring, pos
    return out, final_state


def _check_decode(q, k, v, state, ring, pos, out, per_head: bool):
    if q.dim() != 3 or k.dim() != 3 or ring.dim() != 5:
        raise ValueError("q must be [B, Hq, d], k and v [B, Hkv, d], ring [B, Hkv, 2, w, d]")
    B, Hq, d = q.shape
    Hkv = k.shape[1]
    w = ring.shape[3]
    _expect(k, "k", (B, Hkv, d), q.dtype)
    _expect(v, "v", (B, Hkv, d), q.dtype)
    _expect(state, "state", (B, Hq if per_head else Hkv, d, d), torch.float32)
    _expect(ring, "ring", (B, Hkv, 2, w, d), q.dtype)
    _expect(pos, "pos", (B,), torch.int32)
    _expect(out, "out", (B, Hq, d), q.dtype)
    _need_cuda(q, k, v, state, ring, pos, out)
    return B, Hq, Hkv, d, w


def decode(q, k, v, state, ring, pos, alpha: float = 0.5, out=None, stream=None):
    """One Liger Attention decode step; updates state, ring and pos in place.

    q [B, Hq, d], k and v [B, Hkv, d]; state [B, Hq, d, d] fp32; ring
    [B, Hkv, 2, w, d]; pos [B] int32.  Returns out [B, Hq, d].
    """
    lib = load()
    B, Hq, Hkv, d, w = _check_decode(q, k, v, state, ring, pos, out, per_head=True)
    if out is None:
        out = torch.empty_like(q)
    st = lib.liger_attn_decode(
        _ptr(q), _ptr(k), _ptr(v), _ptr(state), _ptr(ring), _ptr(out), _ptr(pos), B, Hq, Hkv, d, w,
        float(alpha), _dt(q), _stream_ptr(stream))
    _check(st)
    return out


def decode_kvshared(q, k, v, state, ring, pos, alpha: float = 0.5, out=None, stream=None):
    """One decode step over one state per (sequence, kv head): state [B, Hkv, d, d] fp32.

    Equivalent to `decode` when the per-head states of each group are equal (as
    prefill leaves them); moves G = Hq/Hkv times less state per step.
    """
    lib = load()
    B, Hq, Hkv, d, w = _check_decode(q, k, v, state, ring, pos, out, per_head=False)
    if out is None:
        out = torch.empty_like(q)
    st = lib.liger_attn_decode_kvshared(
        _ptr(q), _ptr(k), _ptr(v), _ptr(state), _ptr(ring), _ptr(out), _ptr(pos), B, Hq, Hkv, d, w,
        float(alpha), _dt(q), _stream_ptr(stream))
    _check(st)
    return out


def prefill_status(workspace) -> int:
    """LIGER_OK, or LIGER_ERR_TIMEOUT if the last prefill on this workspace gave up waiting
    (call after its stream has completed)."""
    if workspace is None:
        return LIGER_OK
    return int(load().liger_attn_prefill_status(_ptr(workspace), workspace.numel() * workspace.element_size()))


def full_causal_attention(q, k, v, cu_seqlens=None, max_seqlen=None, out=None, stream=None):
    """Causal softmax attention (the hybrid's standard attention layer), bf16.

    q [B, T, Hq, d], k and v [B, T, Hkv, d]; cu_seqlens as for `prefill` (B must be 1), with
    max_seqlen the longest sequence (computed from cu_seqlens when not given, which reads it
    back to the host).  Returns out [B, T, Hq, d].
    """
    lib = load()
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B, T, Hq, d] and k, v [B, T, Hkv, d]")
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    _expect(k, "k", (B, T, Hkv, d), q.dtype)
    _expect(v, "v", (B, T, Hkv, d), q.dtype)
    _expect(out, "out", (B, T, Hq, d), q.dtype)
    if cu_seqlens is not None and (cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2
                                   or cu_seqlens.dtype != torch.int32):
        raise ValueError("cu_seqlens must be a 1-D int32 tensor of n + 1 offsets")
    _need_cuda(q, k, v, out, cu_seqlens)
    n = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if cu_seqlens is not None and max_seqlen is None:
        max_seqlen = int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item())
    if out is None:
        out = torch.empty_like(q)
    st = lib.liger_attn_full_causal(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, Hq, Hkv, T, d, _dt(q),
                                    _ptr(cu_seqlens), n, 0 if max_seqlen is None else int(max_seqlen),
                                    _stream_ptr(stream))
    _check(st)
    return out


def full_causal_status() -> int:
    """LIGER_OK, or LIGER_ERR_TIMEOUT if a causal attention call gave up waiting since the last query."""
    return int(load().liger_attn_full_causal_status())


def decode_status() -> int:
    """LIGER_OK, or LIGER_ERR_TIMEOUT if a decode step gave up waiting since the last query."""
    return int(load().liger_attn_decode_status())


def prefill_backward_workspace_size(B, Hq, Hkv, T, d, n_seqs, dtype=torch.bfloat16) -> int:
    return int(load().liger_attn_prefill_backward_workspace_size(
        B, Hq, Hkv, T, d, n_seqs, LIGER_BF16 if dtype == torch.bfloat16 else LIGER_FP32))


def prefill_backward(q, k, v, d_out, alpha: float = 0.5, w: int = 64, d_final_state=None,
                     initial_state=None, cu_seqlens=None, want_d_initial_state: bool = False,
                     workspace=None, stream=None):
    """Gradient of `prefill` for L = sum(d_out * out) + sum(d_final_state * final_state).

    initial_state and the returned d_initial_state are one per (sequence, kv head):
    [n, Hkv, d, d] fp32.  Returns (dq, dk, dv, d_initial_state or None).
    """
    lib = load()
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B, T, Hq, d] and k, v [B, T, Hkv, d]")
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    _expect(k, "k", (B, T, Hkv, d), q.dtype)
    _expect(v, "v", (B, T, Hkv, d), q.dtype)
    _expect(d_out, "d_out", (B, T, Hq, d), q.dtype)
    if cu_seqlens is not None and (cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2
                                   or cu_seqlens.dtype != torch.int32):
        raise ValueError("cu_seqlens must be a 1-D int32 tensor of n + 1 offsets")
    n = B if cu_seqlens is None else cu_seqlens.numel() - 1
    _expect(d_final_state, "d_final_state", (n, Hq, d, d), torch.float32)
    _expect(initial_state, "initial_state", (n, Hkv, d, d), torch.float32)
    _need_cuda(q, k, v, d_out, d_final_state, initial_state, cu_seqlens, workspace)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ds0 = torch.empty(n, Hkv, d, d, device=q.device, dtype=torch.float32) if want_d_initial_state else None
    need = prefill_backward_workspace_size(B, Hq, Hkv, T, d, n, q.dtype)
    if workspace is None and need:
        workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.liger_attn_prefill_backward(
        _ptr(q), _ptr(k), _ptr(v), _ptr(d_out), _ptr(d_final_state), _ptr(initial_state), B, Hq, Hkv, T, d, w,
        float(alpha), _dt(q), _ptr(cu_seqlens), n, _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ds0), _ptr(workspace),
        ws_bytes, _stream_ptr(stream))
    _check(st)
    return dq, dk, dv, ds0


def prefill_vector_gate_workspace_size(B, Hq, Hkv, T, d, n_seqs, dtype=torch.bfloat16) -> int:
    return int(load().liger_attn_prefill_vector_gate_workspace_size(
        B, Hq, Hkv, T, d, n_seqs, LIGER_BF16 if dtype == torch.bfloat16 else LIGER_FP32))


def prefill_vector_gate(q, k, v, alpha: float = 0.5, w: int = 64, initial_state=None, cu_seqlens=None,
                        return_ring: bool = False, workspace=None, stream=None):
    """The prefill with one gate per key dimension (sigmoid(k_t[r]) on row r of the state).
    Returns (out, final_state) or, with return_ring, (out, final_state, ring, pos).
    workspace: uint8 CUDA tensor of prefill_vector_gate_workspace_size() bytes (allocated
    here when None)."""
    lib = load()
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B, T, Hq, d] and k, v [B, T, Hkv, d]")
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    _expect(k, "k", (B, T, Hkv, d), q.dtype)
    _expect(v, "v", (B, T, Hkv, d), q.dtype)
    if cu_seqlens is not None and (cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2
                                   or cu_seqlens.dtype != torch.int32):
        raise ValueError("cu_seqlens must be a 1-D int32 tensor of n + 1 offsets")
    n = B if cu_seqlens is None else cu_seqlens.numel() - 1
    _expect(initial_state, "initial_state", (n, Hq, d, d), torch.float32)
    _need_cuda(q, k, v, initial_state, cu_seqlens)
    out = torch.empty_like(q)
    fs = torch.empty(n, Hq, d, d, device=q.device, dtype=torch.float32)
    ring = torch.empty(n, Hkv, 2, w, d, device=q.device, dtype=q.dtype) if return_ring else None
    pos = torch.empty(n, device=q.device, dtype=torch.int32) if return_ring else None
    need = lib.liger_attn_prefill_vector_gate_workspace_size(B, Hq, Hkv, T, d, n, _dt(q))
    if workspace is None:
        workspace = torch.empty(max(need, 1), device=q.device, dtype=torch.uint8)
    _need_cuda(workspace)
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    st = lib.liger_attn_prefill_vector_gate(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(fs), B, Hq, Hkv, T, d, w, float(alpha), _dt(q),
        _ptr(initial_state), _ptr(cu_seqlens), n, _ptr(ring), _ptr(pos), _ptr(workspace), workspace.numel(),
        _stream_ptr(stream))
    _check(st)
    return (out, fs, ring, pos) if return_ring else (out, fs)


def decode_vector_gate(q, k, v, state, ring, pos, alpha: float = 0.5, out=None, stream=None):
    """One decode step with one gate per key dimension; updates state, ring and pos in place."""
    lib = load()
    B, Hq, Hkv, d, w = _check_decode(q, k, v, state, ring, pos, out, per_head=True)
    if out is None:
        out = torch.empty_like(q)
    st = lib.liger_attn_decode_vector_gate(
        _ptr(q), _ptr(k), _ptr(v), _ptr(state), _ptr(ring), _ptr(out), _ptr(pos), B, Hq, Hkv, d, w,
        float(alpha), _dt(q), _stream_ptr(stream))
    _check(st)
    return out


# ------------------------------------------------------------------ paged 8-bit cache

def _kv_dt(cache: torch.Tensor) -> int:
    if cache.dtype == torch.float8_e4m3fn:
        return LIGER_KV_E4M3
    if cache.dtype == torch.int8:
        return LIGER_KV_INT8
    raise TypeError(f"unsupported cache dtype {cache.dtype} (float8_e4m3fn or int8)")


def _elsewhere(dev, stream):
    """What a call enters first if it runs on another stream than the current one, or on another device than the
    current one (launches go to the tensors' device, and what a call allocates belongs to the stream it runs
    on); None if nothing is to be entered."""
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
        return torch.cuda.stream(stream)   # (makes dev current as well)
    return None if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _current_raw_stream(dev) -> int:
    # (torch.cuda.current_stream() costs two microseconds, a third of a launch)
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _need_cuda_strided(*ts):
    """As _need_cuda, for tensors whose layout has been checked apart.  Returns their device."""
    at = ts[0].get_device()   # (-1 on the host)
    for t in ts:
        if t is not None and (at < 0 or t.get_device() != at):
            if not t.is_cuda:
                raise ValueError("tensors must be CUDA tensors")
            raise ValueError(f"tensors must be on one device ({ts[0].device} and {t.device})")
    return ts[0].device


def _token_stride(t, name, heads, d):
    """Elements between the tokens of [..., heads, d], heads and elements contiguous, the tokens
    evenly spaced (a slice of a fused projection, for instance)."""
    if t.is_contiguous():
        return heads * d
    sh, st = t.shape, t.stride()
    ok = (d == 1 or st[-1] == 1) and (heads == 1 or st[-2] == d)
    lead = [(n, s) for n, s in zip(sh[:-2], st[:-2]) if n > 1]
    for (_, outer), (n, inner) in zip(lead, lead[1:]):
        ok = ok and outer == n * inner
    if not ok:
        raise ValueError(f"{name}: heads and elements must be contiguous and tokens evenly spaced, got strides {tuple(st)}")
    return lead[-1][1] if lead else heads * d


def _check_cache(cache, scales):
    if cache.dim() != 5 or cache.shape[2] != 2:
        raise ValueError("cache must be [n_blocks, Hkv, 2, block_size, d]")
    n_blocks, Hkv, _, block_size, d = cache.shape
    _expect(scales, "scales", (n_blocks, Hkv, 2), torch.float32)
    if not cache.is_contiguous() or not scales.is_contiguous():
        raise ValueError("cache and scales must be contiguous")
    return n_blocks, Hkv, block_size, d, _kv_dt(cache)


def kv_cache_new(n_blocks: int, Hkv: int, d: int, block_size: int, max_seqs: int, max_tokens: int,
                 dtype=torch.float8_e4m3fn, device="cuda") -> dict:
    """The tensors of an empty paged 8-bit cache for max_seqs sequences of up to max_tokens tokens.

    cache [n_blocks, Hkv, 2, block_size, d] (e4m3 or int8), scales [n_blocks, Hkv, 2] fp32, block_table
    [max_seqs, ceil(max_tokens / block_size)], seq_lens [max_seqs], free_blocks [n_blocks] and free_span [2]
    (int32): all blocks free.
    """
    i32 = dict(device=device, dtype=torch.int32)
    cache = torch.zeros(n_blocks, Hkv, 2, block_size, d, device=device, dtype=torch.uint8).view(dtype)
    _kv_dt(cache)
    return {"cache": cache, "scales": torch.ones(n_blocks, Hkv, 2, device=device, dtype=torch.float32),
            "block_table": torch.full((max_seqs, -(-max_tokens // block_size)), -1, **i32),
            "seq_lens": torch.zeros(max_seqs, **i32), "free_blocks": torch.arange(n_blocks, **i32),
            "free_span": torch.tensor([0, n_blocks], **i32)}


def kv_cache_assign(new_lens, seq_lens, block_table, free_blocks, free_span, block_size: int, n_slots: int,
                    slot_map=None, cu_new=None, seq_lens_out=None, free_span_out=None, stream=None):
    """Block tables and slot maps from request lengths (int32 CUDA tensors, all on the device).

    new_lens [B]: tokens to add to each sequence; a negative number ends it and gives its blocks
    back.  seq_lens [B], block_table [B, width], free_blocks [n_blocks] and free_span [2]: the state
    (`kv_cache_new`); the table and the ring of free blocks are updated in place.  n_slots: length of the
    slot map (at least the sum of the new lengths; the rest is -1).  seq_lens_out and free_span_out may be
    seq_lens and free_span (the state then advances in place).  Returns (slot_map [n_slots], cu_new [B + 1],
    seq_lens_out, free_span_out).

    Lengths only grow, or end: do not lower seq_lens over a block border, the blocks behind it would be
    lost.  Where drafted tokens may be turned down, assign all of them into new seq_lens_out and
    free_span_out, append and attend; then assign the kept ones from the same seq_lens and free_span
    as before, and append those again.
    """
    lib = load()
    if new_lens.dim() != 1 or block_table.dim() != 2 or free_blocks.dim() != 1:
        raise ValueError("new_lens must be [B], block_table [B, width] and free_blocks [n_blocks]")
    B, i32 = new_lens.shape[0], torch.int32
    if new_lens.dtype != i32 or free_blocks.dtype != i32:
        raise ValueError("new_lens and free_blocks must be int32")
    width, n_blocks = block_table.shape[1], free_blocks.shape[0]
    _expect(seq_lens, "seq_lens", (B,), i32)
    _expect(block_table, "block_table", (B, width), i32)
    _expect(free_span, "free_span", (2,), i32)
    _expect(slot_map, "slot_map", (n_slots,), i32)
    _expect(cu_new, "cu_new", (B + 1,), i32)
    _expect(seq_lens_out, "seq_lens_out", (B,), i32)
    _expect(free_span_out, "free_span_out", (2,), i32)
    tensors = (new_lens, seq_lens, block_table, free_blocks, free_span, slot_map, cu_new, seq_lens_out, free_span_out)
    for t in tensors:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")
    dev = _need_cuda_strided(*tensors)
    on = _elsewhere(dev, stream)
    if on is not None:
        with on:
            return kv_cache_assign(new_lens, seq_lens, block_table, free_blocks, free_span, block_size, n_slots, slot_map,
                                   cu_new, seq_lens_out, free_span_out)
    if slot_map is None:
        slot_map = torch.empty(n_slots, device=dev, dtype=i32)
    if cu_new is None:
        cu_new = torch.empty(B + 1, device=dev, dtype=i32)
    if seq_lens_out is None:
        seq_lens_out = torch.empty_like(seq_lens)
    if free_span_out is None:
        free_span_out = torch.empty_like(free_span)
    st = lib.liger_kv_cache_assign(
        new_lens.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(), free_blocks.data_ptr(), free_span.data_ptr(),
        slot_map.data_ptr(), cu_new.data_ptr(), seq_lens_out.data_ptr(), free_span_out.data_ptr(), B, width, n_blocks,
        block_size, n_slots, _current_raw_stream(dev))
    _check(st)
    return slot_map, cu_new, seq_lens_out, free_span_out


def kv_cache_append(k, v, slot_map, cache, scales, stream=None):
    """Quantises keys and values into their slots of the cache (in place).

    k, v [N, Hkv, d] (bf16 or fp32; tokens may be evenly strided), slot_map [N] int32 as
    `kv_cache_assign` gives it (-1: left out), cache [n_blocks, Hkv, 2, block_size, d], scales
    [n_blocks, Hkv, 2] fp32.
    """
    lib = load()
    n_blocks, Hkv, block_size, d, kv_dt = _check_cache(cache, scales)
    if k.dim() != 3:
        raise ValueError("k and v must be [N, Hkv, d]")
    N = k.shape[0]
    _expect(k, "k", (N, Hkv, d), k.dtype)
    _expect(v, "v", (N, Hkv, d), k.dtype)
    _expect(slot_map, "slot_map", (N,), torch.int32)
    if not slot_map.is_contiguous():
        raise ValueError("slot_map must be contiguous")
    dt = _dt(k)
    ks, vs = _token_stride(k, "k", Hkv, d), _token_stride(v, "v", Hkv, d)
    dev = _need_cuda_strided(k, v, slot_map, cache, scales)
    on = _elsewhere(dev, stream)
    if on is not None:
        with on:
            return kv_cache_append(k, v, slot_map, cache, scales)
    st = lib.liger_kv_cache_append(k.data_ptr(), v.data_ptr(), slot_map.data_ptr(), cache.data_ptr(), scales.data_ptr(),
                                   N, Hkv, d, n_blocks, block_size, ks, vs, dt, kv_dt, _current_raw_stream(dev))
    _check(st)


def cached_attention_workspace_size(d: int) -> int:
    """Bytes of workspace of cached_attention on the current device."""
    return int(load().liger_attn_cached_workspace_size(d))


@functools.lru_cache(maxsize=None)
def _cached_workspace(device: int, d: int) -> int:
    return cached_attention_workspace_size(d)


def cached_attention(q, cache, scales, block_table, seq_lens, out=None, workspace=None, stream=None):
    """Softmax attention of each sequence's newest tokens over its cached tokens, themselves
    included (one decode step of the hybrid's standard attention layer).

    q [B, Hq, d], or [B, n_q, Hq, d] for n_q <= 16 new tokens a sequence (bf16 or fp32; tokens may be
    evenly strided); cache, scales, block_table [B, width] and seq_lens [B] as for `kv_cache_append`, seq_lens
    with the new tokens counted.  Query i is the token len - n_q + i: a sequence with fewer new tokens has
    their queries last, and the rows before them can be left aside (zeros before its first token).  fp32
    queries and weights keep 22 bits (two fp16 terms), bf16 calls round weights to fp16.
    workspace: uint8 CUDA tensor of cached_attention_workspace_size(d)
    bytes (allocated here when None).  Returns out in q's shape.
    """
    lib = load()
    n_blocks, Hkv, block_size, d, kv_dt = _check_cache(cache, scales)
    shape = q.shape
    if len(shape) not in (3, 4) or shape[-1] != d:
        raise ValueError(f"q must be [B, Hq, {d}] or [B, n_q, Hq, {d}]")
    if block_table.dim() != 2 or block_table.dtype != torch.int32:
        raise ValueError("block_table must be [B, width] int32")
    B, Hq = shape[0], shape[-2]
    n_q = shape[1] if len(shape) == 4 else 1
    width = block_table.shape[1]
    _expect(block_table, "block_table", (B, width), torch.int32)
    _expect(seq_lens, "seq_lens", (B,), torch.int32)
    _expect(out, "out", shape, q.dtype)
    dt = _dt(q)
    qs = _token_stride(q, "q", Hq, d)
    if not (block_table.is_contiguous() and seq_lens.is_contiguous() and (out is None or out.is_contiguous())
            and (workspace is None or workspace.is_contiguous())):
        raise ValueError("block_table, seq_lens, out and workspace must be contiguous")
    dev = _need_cuda_strided(q, cache, scales, block_table, seq_lens, out, workspace)
    on = _elsewhere(dev, stream)
    if on is not None:
        with on:
            return cached_attention(q, cache, scales, block_table, seq_lens, out, workspace)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if workspace is None:
        workspace = torch.empty(_cached_workspace(dev.index, d), device=dev, dtype=torch.uint8)
    st = lib.liger_attn_cached(
        q.data_ptr(), cache.data_ptr(), scales.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), out.data_ptr(),
        B, n_q, Hq, Hkv, d, width, n_blocks, block_size, qs, dt, kv_dt, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _current_raw_stream(dev))
    _check(st)
    return out


def cached_attention_status() -> int:
    """LIGER_OK, or LIGER_ERR_TIMEOUT if a cached attention call gave up waiting since the last query."""
    return int(load().liger_attn_cached_status())
