"""Python binding of the C ABI in ``include/fa_gb300.h`` (ctypes).

Argument marshalling only: tensors become device pointers, the stream becomes
a ``cudaStream_t``; every step of the computation runs in the CUDA library.
There is no fallback: if the library is missing or cannot be loaded, every
call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

from . import build as _build

_LIB: Optional[ctypes.CDLL] = None

FA_OK = 0
FA_ERR_INVALID = -1
FA_ERR_UNSUPPORTED = -2
FA_ERR_LAUNCH = -3
FA_ERR_TIMEOUT = -4
FA_ERR_WORKSPACE = -5
FA_ERR_SCRATCH_LIMIT = -6
NOALLOC_SCRATCH_BYTES = 64 << 20

# Every symbol the header declares, with its ctypes signature.
_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_L = ctypes.c_longlong
SIGNATURES = {
    "fa_fwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _P, _P]),
    "fa_fwd_varlen": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    "fa_bwd_workspace_size": (ctypes.c_size_t, [_I, _I, _I, _I]),
    "fa_decode_workspace_size": (ctypes.c_size_t, [_I, _I, _I, _I]),
    "fa_quantize_fp8": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "fa_fwd_fp8": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _P, _P]),
    "fa_decode_paged": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, ctypes.c_size_t, _P]),
    "fa_bwd_varlen": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P,
                           ctypes.c_size_t, _P]),
    "fa_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _P, _P, ctypes.c_size_t, _P]),
    "fa_bwd_deterministic": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _P, _P,
                                  ctypes.c_size_t, _P]),
    "fa_bwd_varlen_deterministic": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I,
                                         _F, _I, _P, ctypes.c_size_t, _P]),
    "fa_fwd_varlen_gqa": (_I, [_P] * 7 + [_I] * 8 + [_F, _I, _P]),
    "fa_bwd_varlen_gqa": (_I, [_P] * 11 + [_I] * 8 + [_F, _I, _P, ctypes.c_size_t, _P]),
    "fa_bwd_varlen_gqa_deterministic": (_I, [_P] * 11 + [_I] * 8 + [_F, _I, _P, ctypes.c_size_t, _P]),
    "fa_qk_norm_rope": (_I, [_P] * 9 + [_I] * 6 + [_L, _L, _F, _I, _P]),
    "fa_qk_norm_rope_bwd_workspace_size": (ctypes.c_size_t, [_I, _I, _I, _I]),
    "fa_qk_norm_rope_bwd": (_I, [_P] * 13 + [_I] * 6 + [_L] * 4 + [_F, _I, _P, ctypes.c_size_t, _P]),
    "fa_decode_shared_prefix_workspace_size": (ctypes.c_size_t, [_I] * 8),
    "fa_decode_shared_prefix": (_I, [_P] * 10 + [_I] * 12 + [_F, _P, ctypes.c_size_t, _P]),
    "fa_kv_append": (_I, [_P] * 10 + [_I] * 8 + [_L, _L, _L, _I, _P]),
    "fa_kv_append_q4": (_I, [_P] * 12 + [_I] * 8 + [_L, _L, _L, _I, _P]),
    "fa_kv_gather_q4": (_I, [_P] * 9 + [_I] * 7 + [_P]),
    "fa_decode_paged_q4_workspace_size": (ctypes.c_size_t, [_I] * 6),
    "fa_decode_paged_q4": (_I, [_P] * 9 + [_I] * 9 + [_F, _P, ctypes.c_size_t, _P]),
    "fa_check_status": (_I, [_P]),
    "fa_status_string": (ctypes.c_char_p, [_I]),
    "fa_last_cuda_error": (ctypes.c_char_p, []),
    "fa_bwd_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _P, _P]),
    "fa_timing_begin": (_I, [_I]),
    "fa_timing_read": (_I, [_I, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int)]),
    "fa_timing_end": (_I, []),
}

(KERNEL_FWD, KERNEL_BWD_PRE, KERNEL_BWD_MAIN, KERNEL_BWD_DQ, KERNEL_DECODE, KERNEL_DECODE_MERGE,
 KERNEL_FWD_FP8) = range(7)


class FaError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = load_library()
        msg = lib.fa_status_string(status).decode()
        if status == FA_ERR_LAUNCH:
            msg += " (" + lib.fa_last_cuda_error().decode() + ")"
        super().__init__(f"{where}: {msg}")
        self.status = status


def library_path() -> str:
    return _build.LIB


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load the CUDA library (raises if it has not been built)."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    p = path or _build.LIB
    if not os.path.exists(p):
        raise RuntimeError(f"CUDA attention library not built ({p}); run exact_io_aware_29_gb300.build.build()")
    lib = ctypes.CDLL(p)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _LIB = lib
    return lib


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _check_bhnd(name, t, shape=None):
    import torch
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16")
    if t.dim() != 4 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name} must have shape [B, H, N, d] = {shape}")


def fa_fwd(q, k, v, o, lse, scale: float, causal: bool, kv_lens=None, stream=None) -> None:
    """O, LSE <- attention(Q, K, V); same semantics as the C entry point."""
    import torch
    _check_bhnd("q", q)
    B, H, N, d = q.shape
    for name, t in (("k", k), ("v", v), ("o", o)):
        _check_bhnd(name, t, q.shape)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [B, H, N] CUDA tensor")
    if kv_lens is not None and (kv_lens.dtype != torch.int32 or not kv_lens.is_cuda or kv_lens.numel() != B):
        raise ValueError("kv_lens must be an int32 [B] CUDA tensor")
    st = load_library().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, float(scale),
                               int(bool(causal)), _ptr(kv_lens), _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_fwd")


def _check_thd(name, t, H=None, d=None):
    import torch
    if not t.is_cuda or not t.is_contiguous() or t.dtype != torch.bfloat16 or t.dim() != 3:
        raise ValueError(f"{name} must be a contiguous bfloat16 CUDA tensor [total, H, d]")
    if (H is not None and t.shape[1] != H) or (d is not None and t.shape[2] != d):
        raise ValueError(f"{name} has the wrong H or d")


def _check_cu(name, cu, batch=None):
    import torch
    if cu.dtype != torch.int32 or not cu.is_cuda or cu.dim() != 1 or (batch is not None and cu.numel() != batch + 1):
        raise ValueError(f"{name} must be an int32 CUDA tensor [batch + 1]")


def fa_fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int,
                  scale: float, causal: bool, stream=None) -> None:
    """Packed variable-length forward; same semantics as the C entry point."""
    import torch
    _check_thd("q", q)
    total_q, H, d = q.shape
    _check_thd("k", k, H, d)
    _check_thd("v", v, H, d)
    _check_thd("o", o, H, d)
    if tuple(o.shape) != tuple(q.shape) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("o must match q and v must match k")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (H, total_q) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [H, total_q] CUDA tensor")
    _check_cu("cu_seqlens_q", cu_seqlens_q)
    batch = cu_seqlens_q.numel() - 1
    _check_cu("cu_seqlens_k", cu_seqlens_k, batch)
    st = load_library().fa_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(cu_seqlens_q),
                                      _ptr(cu_seqlens_k), batch, H, d, total_q, k.shape[0], int(max_seqlen_q),
                                      int(max_seqlen_k), float(scale), int(bool(causal)), _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_fwd_varlen")


def attention_forward_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale, causal,
                             stream=None):
    """Allocates O [total_q, H, d] and LSE [H, total_q], then calls fa_fwd_varlen."""
    import torch
    o = torch.empty_like(q)
    lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
    fa_fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale, causal, stream)
    return o, lse


def fa_bwd_varlen(q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                  max_seqlen_k: int, scale: float, causal: bool, workspace=None, stream=None) -> None:
    """Packed variable-length backward; same semantics as the C entry point."""
    _bwd_varlen("fa_bwd_varlen", q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                max_seqlen_k, scale, causal, workspace, stream)


def fa_bwd_varlen_deterministic(q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                                max_seqlen_k: int, scale: float, causal: bool, workspace=None,
                                stream=None) -> None:
    """fa_bwd_varlen with dQ summed in a fixed order: bitwise reproducible results."""
    _bwd_varlen("fa_bwd_varlen_deterministic", q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens_q, cu_seqlens_k,
                max_seqlen_q, max_seqlen_k, scale, causal, workspace, stream)


def _bwd_varlen(fn, q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
                scale, causal, workspace, stream) -> None:
    import torch
    _check_thd("q", q)
    total_q, H, d = q.shape
    for name, t in (("k", k), ("v", v), ("o", o), ("dO", dO), ("dq", dq), ("dk", dk), ("dv", dv)):
        _check_thd(name, t, H, d)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (H, total_q):
        raise ValueError("lse must be float32 [H, total_q]")
    _check_cu("cu_seqlens_q", cu_seqlens_q)
    batch = cu_seqlens_q.numel() - 1
    _check_cu("cu_seqlens_k", cu_seqlens_k, batch)
    need = fa_bwd_workspace_size(batch, H, int(max_seqlen_q), d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    st = getattr(load_library(), fn)(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq),
                                     _ptr(dk), _ptr(dv), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), batch, H, d,
                                     total_q, k.shape[0], int(max_seqlen_q), int(max_seqlen_k), float(scale),
                                     int(bool(causal)), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _stream(stream))
    if st != FA_OK:
        raise FaError(st, fn)


def attention_backward_varlen(q, k, v, o, lse, dO, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
                              scale, causal, workspace=None, stream=None, deterministic: bool = False):
    """Allocates dQ, dK, dV, then calls fa_bwd_varlen (or its deterministic
    form). Returns (dQ, dK, dV)."""
    import torch
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    fn = fa_bwd_varlen_deterministic if deterministic else fa_bwd_varlen
    fn(q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale, causal,
       workspace, stream)
    return dq, dk, dv


# ---------------------------------------------------------------------------
# The grouped-head operators are called once per layer and token, where the
# host's time counts: a call checks its tensors in one expression, and only a
# call that fails it goes over them by name.
# ---------------------------------------------------------------------------
_torch = None


def _load_torch():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _refuse(where, dev, wanted) -> None:
    """Raises for the first (name, tensor, dtype, shape) that is not
    contiguous, of that dtype and shape, on CUDA device ``dev``."""
    for name, t, dtype, shape in wanted:
        if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
            raise ValueError(f"{where}: {name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                             f"cuda:{dev}; got {t.dtype} {tuple(t.shape)} on {t.device}" +
                             ("" if t.is_contiguous() else ", strided"))
    raise ValueError(f"{where}: arguments do not fit together")


def _cuda_index(where, t) -> int:
    dev = t.get_device()
    if dev < 0 or not t.is_cuda:
        raise ValueError(f"{where} needs CUDA tensors")
    return dev


def _raw_stream(where, dev, stream):
    """The cudaStream_t of a call on device ``dev`` (None: its current stream)."""
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(dev)
    if stream.device.index != dev:
        raise ValueError(f"{where}: the stream belongs to {stream.device}, the tensors to cuda:{dev}")
    return stream.cuda_stream


def _on_device(dev, fn, *args):
    """fn(*args) with device ``dev`` current (the library launches on the current device)."""
    if dev == _torch._C._cuda_getDevice():
        return fn(*args)
    with _torch.cuda.device(dev):
        return fn(*args)


def _alloc(stream, make):
    """make() with the tensors belonging to the stream that the call runs on:
    what another stream may still be using is not handed to it, and what it
    uses is not handed to another one when the tensor dies."""
    if stream is None:
        return make()
    with _load_torch().cuda.stream(stream):
        return make()


def _workspace(where, t, dev, stream, size, *sizes):
    """The caller's workspace, or one of size(*sizes) bytes."""
    if t is None:
        return _alloc(stream, lambda: _torch.empty(max(size(*sizes), 1), dtype=_torch.uint8, device=f"cuda:{dev}"))
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{where}: workspace must be a contiguous tensor on cuda:{dev}")
    return t


def _check_gqa(where, q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k):
    """Checks what both directions of the grouped-head packed attention take:
    (device, the C call's sizes up to total_k)."""
    torch = _torch or _load_torch()
    dev = _cuda_index(where, q)
    qs, ks, bf16, i32 = q.shape, k.shape, torch.bfloat16, torch.int32
    if len(qs) != 3 or len(ks) != 3 or ks[2] != qs[2] or ks[1] < 1 or qs[1] % ks[1]:
        raise ValueError(f"{where}: q is [total_q, H, d], k and v [total_k, H_kv, d] with H a multiple of H_kv; got "
                         f"{tuple(qs)} and {tuple(ks)}")
    total_q, H, d = qs
    n = cu_seqlens_q.numel()
    if (q.dtype is not bf16 or not q.is_contiguous()
            or k.dtype is not bf16 or not k.is_contiguous() or k.get_device() != dev
            or v.dtype is not bf16 or v.shape != ks or not v.is_contiguous() or v.get_device() != dev
            or o.dtype is not bf16 or o.shape != qs or not o.is_contiguous() or o.get_device() != dev
            or lse.dtype is not torch.float32 or lse.shape != (H, total_q) or not lse.is_contiguous()
            or lse.get_device() != dev
            or cu_seqlens_q.dtype is not i32 or cu_seqlens_q.dim() != 1 or not cu_seqlens_q.is_contiguous()
            or cu_seqlens_q.get_device() != dev
            or cu_seqlens_k.dtype is not i32 or cu_seqlens_k.shape != (n,) or not cu_seqlens_k.is_contiguous()
            or cu_seqlens_k.get_device() != dev):
        _refuse(where, dev, (("q", q, bf16, qs), ("k", k, bf16, ks), ("v", v, bf16, ks), ("o", o, bf16, qs),
                             ("lse", lse, torch.float32, (H, total_q)), ("cu_seqlens_q", cu_seqlens_q, i32, (n,)),
                             ("cu_seqlens_k", cu_seqlens_k, i32, (n,))))
    return dev, (n - 1, H, ks[1], d, total_q, ks[0])


def fa_fwd_varlen_gqa(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int,
                      scale: float, causal: bool, stream=None) -> None:
    """Packed forward with grouped heads (q [total_q, H, d], k and v
    [total_k, H_kv, d]); same semantics as the C entry point."""
    where = "fa_fwd_varlen_gqa"
    dev, sizes = _check_gqa(where, q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k)
    st = _on_device(dev, (_LIB or load_library()).fa_fwd_varlen_gqa, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                    o.data_ptr(), lse.data_ptr(), cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), *sizes,
                    int(max_seqlen_q), int(max_seqlen_k), float(scale), int(bool(causal)),
                    _raw_stream(where, dev, stream))
    if st != FA_OK:
        raise FaError(st, where)


def attention_forward_varlen_gqa(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale, causal,
                                 stream=None):
    """Allocates O [total_q, H, d] and LSE [H, total_q], then calls fa_fwd_varlen_gqa."""
    torch = _load_torch()
    o, lse = _alloc(stream, lambda: (torch.empty_like(q), torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32,
                                                                      device=q.device)))
    fa_fwd_varlen_gqa(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale, causal, stream)
    return o, lse


def _bwd_varlen_gqa(fn, q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
                    scale, causal, workspace, stream) -> None:
    dev, sizes = _check_gqa(fn, q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k)
    qs, ks, bf16 = q.shape, k.shape, _torch.bfloat16
    if (dO.dtype is not bf16 or dO.shape != qs or not dO.is_contiguous() or dO.get_device() != dev
            or dq.dtype is not bf16 or dq.shape != qs or not dq.is_contiguous() or dq.get_device() != dev
            or dk.dtype is not bf16 or dk.shape != ks or not dk.is_contiguous() or dk.get_device() != dev
            or dv.dtype is not bf16 or dv.shape != ks or not dv.is_contiguous() or dv.get_device() != dev):
        _refuse(fn, dev, (("dO", dO, bf16, qs), ("dq", dq, bf16, qs), ("dk", dk, bf16, ks), ("dv", dv, bf16, ks)))
    workspace = _workspace(fn, workspace, dev, stream, fa_bwd_workspace_size, sizes[0], sizes[1], int(max_seqlen_q),
                           sizes[3])
    st = _on_device(dev, getattr(_LIB or load_library(), fn), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                    lse.data_ptr(), dO.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                    cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), *sizes, int(max_seqlen_q), int(max_seqlen_k),
                    float(scale), int(bool(causal)), workspace.data_ptr(),
                    workspace.numel() * workspace.element_size(), _raw_stream(fn, dev, stream))
    if st != FA_OK:
        raise FaError(st, fn)


def fa_bwd_varlen_gqa(q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                      max_seqlen_k: int, scale: float, causal: bool, workspace=None, stream=None) -> None:
    """Packed backward with grouped heads; same semantics as the C entry point."""
    _bwd_varlen_gqa("fa_bwd_varlen_gqa", q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                    max_seqlen_k, scale, causal, workspace, stream)


def fa_bwd_varlen_gqa_deterministic(q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                                    max_seqlen_k: int, scale: float, causal: bool, workspace=None,
                                    stream=None) -> None:
    """fa_bwd_varlen_gqa with dQ summed in a fixed order: bitwise reproducible results."""
    _bwd_varlen_gqa("fa_bwd_varlen_gqa_deterministic", q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens_q, cu_seqlens_k,
                    max_seqlen_q, max_seqlen_k, scale, causal, workspace, stream)


def attention_backward_varlen_gqa(q, k, v, o, lse, dO, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
                                  scale, causal, workspace=None, stream=None, deterministic: bool = False):
    """Allocates dQ, dK, dV, then calls fa_bwd_varlen_gqa (or its deterministic
    form). Returns (dQ, dK, dV)."""
    torch = _load_torch()
    dq, dk, dv = _alloc(stream, lambda: [torch.empty_like(t) for t in (q, k, v)])
    fn = fa_bwd_varlen_gqa_deterministic if deterministic else fa_bwd_varlen_gqa
    fn(q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale, causal,
       workspace, stream)
    return dq, dk, dv


def fa_bwd_workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(load_library().fa_bwd_workspace_size(B, H, N, d))


def fa_bwd(q, k, v, o, lse, dO, dq, dk, dv, scale: float, causal: bool, kv_lens=None, workspace=None,
           stream=None) -> None:
    """dQ, dK, dV <- gradients of sum(O * dO); same semantics as the C entry point."""
    _bwd_fixed("fa_bwd", q, k, v, o, lse, dO, dq, dk, dv, scale, causal, kv_lens, workspace, stream)


def fa_bwd_deterministic(q, k, v, o, lse, dO, dq, dk, dv, scale: float, causal: bool, kv_lens=None,
                         workspace=None, stream=None) -> None:
    """fa_bwd with dQ summed in a fixed order: bitwise reproducible results."""
    _bwd_fixed("fa_bwd_deterministic", q, k, v, o, lse, dO, dq, dk, dv, scale, causal, kv_lens, workspace, stream)


def _bwd_fixed(fn, q, k, v, o, lse, dO, dq, dk, dv, scale, causal, kv_lens, workspace, stream) -> None:
    import torch
    _check_bhnd("q", q)
    B, H, N, d = q.shape
    for name, t in (("k", k), ("v", v), ("o", o), ("dO", dO), ("dq", dq), ("dk", dk), ("dv", dv)):
        _check_bhnd(name, t, q.shape)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N):
        raise ValueError("lse must be float32 [B, H, N]")
    need = fa_bwd_workspace_size(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    st = getattr(load_library(), fn)(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq),
                                     _ptr(dk), _ptr(dv), B, H, N, d, float(scale), int(bool(causal)),
                                     _ptr(kv_lens), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     _stream(stream))
    if st != FA_OK:
        raise FaError(st, fn)


def fa_bwd_noalloc(q, k, v, o, lse, dO, dq, dk, dv, scale: float, causal: bool, kv_lens=None,
                   stream=None) -> None:
    """fa_bwd with the library's fixed static scratch instead of a workspace:
    for callers that cannot allocate device memory at this point."""
    import torch
    _check_bhnd("q", q)
    B, H, N, d = q.shape
    for name, t in (("k", k), ("v", v), ("o", o), ("dO", dO), ("dq", dq), ("dk", dk), ("dv", dv)):
        _check_bhnd(name, t, q.shape)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N):
        raise ValueError("lse must be float32 [B, H, N]")
    st = load_library().fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq),
                                       _ptr(dk), _ptr(dv), B, H, N, d, float(scale), int(bool(causal)),
                                       _ptr(kv_lens), _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_bwd_noalloc")


def fa_check_status(stream=None) -> int:
    return int(load_library().fa_check_status(_stream(stream)))


def fa_status_string(status: int) -> str:
    return load_library().fa_status_string(status).decode()


def attention_forward(q, k, v, scale: float, causal: bool, kv_lens=None, stream=None):
    """Allocates O and LSE with torch, then calls fa_fwd. Returns (O, LSE)."""
    import torch
    B, H, N, d = q.shape
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    fa_fwd(q, k, v, o, lse, scale, causal, kv_lens, stream)
    return o, lse


def attention_backward(q, k, v, o, lse, dO, scale: float, causal: bool, kv_lens=None, workspace=None,
                       stream=None, deterministic: bool = False):
    """Allocates dQ, dK, dV with torch, then calls fa_bwd (fa_bwd_deterministic
    if ``deterministic``). Returns (dQ, dK, dV)."""
    import torch
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    fn = fa_bwd_deterministic if deterministic else fa_bwd
    fn(q, k, v, o, lse, dO, dq, dk, dv, scale, causal, kv_lens, workspace, stream)
    return dq, dk, dv


def fa_decode_workspace_size(B: int, H: int, d: int, max_seq_len: int) -> int:
    return int(load_library().fa_decode_workspace_size(B, H, d, max_seq_len))


def fa_decode_paged(q, k_cache, v_cache, o, lse, block_table, seq_lens, max_seq_len: int, scale: float,
                    workspace=None, stream=None) -> None:
    """One decoding step over a paged KV cache; same semantics as the C entry point."""
    import torch
    if q.dtype != torch.bfloat16 or q.dim() != 3 or not q.is_contiguous():
        raise ValueError("q must be contiguous bf16 [B, H, d]")
    B, H, d = q.shape
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.dtype != torch.bfloat16 or t.dim() != 4 or tuple(t.shape[2:]) != (H, d) or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous bf16 [num_blocks, block_size, H, d]")
    if tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("k_cache and v_cache must have the same shape")
    if o.dtype != torch.bfloat16 or tuple(o.shape) != (B, H, d) or not o.is_contiguous():
        raise ValueError("o must be contiguous bf16 [B, H, d]")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H):
        raise ValueError("lse must be float32 [B, H]")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != B \
            or not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous int32 [B, max_blocks_per_seq]")
    if seq_lens.dtype != torch.int32 or tuple(seq_lens.shape) != (B,):
        raise ValueError("seq_lens must be int32 [B]")
    num_blocks, block_size = k_cache.shape[:2]
    if workspace is None:
        workspace = torch.empty(max(fa_decode_workspace_size(B, H, d, int(max_seq_len)), 1), dtype=torch.uint8,
                                device=q.device)
    st = load_library().fa_decode_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), _ptr(lse),
                                        _ptr(block_table), _ptr(seq_lens), B, H, d, num_blocks, block_size,
                                        block_table.shape[1], int(max_seq_len), float(scale), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_decode_paged")


def attention_decode_paged(q, k_cache, v_cache, block_table, seq_lens, max_seq_len, scale, workspace=None,
                           stream=None):
    """Allocates O and LSE, then calls fa_decode_paged. Returns (O, LSE)."""
    import torch
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    fa_decode_paged(q, k_cache, v_cache, o, lse, block_table, seq_lens, max_seq_len, scale, workspace, stream)
    return o, lse


def fa_decode_shared_prefix_workspace_size(n_prefix: int, B: int, H: int, H_kv: int, d: int, max_group: int,
                                           max_prefix_len: int, max_seq_len: int) -> int:
    return int(load_library().fa_decode_shared_prefix_workspace_size(n_prefix, B, H, H_kv, d, max_group,
                                                                     max_prefix_len, max_seq_len))


def fa_decode_shared_prefix(q, k_cache, v_cache, o, lse, prefix_table, prefix_lens, cu_prefix_seqs, block_table,
                            seq_lens, max_group: int, max_prefix_len: int, max_seq_len: int, scale: float,
                            workspace=None, stream=None) -> None:
    """One decoding step of sequences that share prefixes, over a paged KV
    cache with grouped heads; same semantics as the C entry point."""
    torch = _torch or _load_torch()
    where = "fa_decode_shared_prefix"
    dev = _cuda_index(where, q)
    qs, cs, bf16, i32 = q.shape, k_cache.shape, torch.bfloat16, torch.int32
    if len(qs) != 3 or len(cs) != 4 or cs[3] != qs[2] or prefix_table.dim() != 2 or block_table.dim() != 2:
        raise ValueError(f"{where}: q is [B, H, d], the caches [num_blocks, block_size, H_kv, d], the tables "
                         f"[rows, blocks per row]; got {tuple(qs)} and {tuple(cs)}")
    B, H, d = qs
    P, prefix_width = prefix_table.shape
    rows, width = block_table.shape
    if (q.dtype is not bf16 or not q.is_contiguous() or rows != B
            or k_cache.dtype is not bf16 or not k_cache.is_contiguous() or k_cache.get_device() != dev
            or v_cache.dtype is not bf16 or v_cache.shape != cs or not v_cache.is_contiguous()
            or v_cache.get_device() != dev
            or o.dtype is not bf16 or o.shape != qs or not o.is_contiguous() or o.get_device() != dev
            or lse.dtype is not torch.float32 or lse.shape != (B, H) or not lse.is_contiguous()
            or lse.get_device() != dev
            or prefix_table.dtype is not i32 or not prefix_table.is_contiguous() or prefix_table.get_device() != dev
            or prefix_lens.dtype is not i32 or prefix_lens.shape != (P,) or not prefix_lens.is_contiguous()
            or prefix_lens.get_device() != dev
            or cu_prefix_seqs.dtype is not i32 or cu_prefix_seqs.shape != (P + 1,)
            or not cu_prefix_seqs.is_contiguous() or cu_prefix_seqs.get_device() != dev
            or block_table.dtype is not i32 or not block_table.is_contiguous() or block_table.get_device() != dev
            or seq_lens.dtype is not i32 or seq_lens.shape != (B,) or not seq_lens.is_contiguous()
            or seq_lens.get_device() != dev):
        _refuse(where, dev, (
            ("q", q, bf16, qs), ("k_cache", k_cache, bf16, cs), ("v_cache", v_cache, bf16, cs), ("o", o, bf16, qs),
            ("lse", lse, torch.float32, (B, H)), ("prefix_table", prefix_table, i32, (P, prefix_width)),
            ("prefix_lens", prefix_lens, i32, (P,)), ("cu_prefix_seqs", cu_prefix_seqs, i32, (P + 1,)),
            ("block_table", block_table, i32, (B, width)), ("seq_lens", seq_lens, i32, (B,))))
    max_group, max_prefix_len, max_seq_len = int(max_group), int(max_prefix_len), int(max_seq_len)
    workspace = _workspace(where, workspace, dev, stream, fa_decode_shared_prefix_workspace_size, P, B, H, cs[2], d,
                           max_group, max_prefix_len, max_seq_len)
    st = _on_device(dev, (_LIB or load_library()).fa_decode_shared_prefix, q.data_ptr(), k_cache.data_ptr(),
                    v_cache.data_ptr(), o.data_ptr(), lse.data_ptr(), prefix_table.data_ptr(),
                    prefix_lens.data_ptr(), cu_prefix_seqs.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
                    P, B, H, cs[2], d, cs[0], cs[1], prefix_width, width, max_group, max_prefix_len, max_seq_len,
                    float(scale), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                    _raw_stream(where, dev, stream))
    if st != FA_OK:
        raise FaError(st, where)


def attention_decode_shared_prefix(q, k_cache, v_cache, prefix_table, prefix_lens, cu_prefix_seqs, block_table,
                                   seq_lens, max_group, max_prefix_len, max_seq_len, scale, workspace=None,
                                   stream=None):
    """Allocates O and LSE, then calls fa_decode_shared_prefix. Returns (O, LSE)."""
    torch = _load_torch()
    o, lse = _alloc(stream, lambda: (torch.empty_like(q),
                                     torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)))
    fa_decode_shared_prefix(q, k_cache, v_cache, o, lse, prefix_table, prefix_lens, cu_prefix_seqs, block_table,
                            seq_lens, max_group, max_prefix_len, max_seq_len, scale, workspace, stream)
    return o, lse


def _heads_stride(where, name, t, T, H, d, dev) -> int:
    """The token stride, in elements, of a bf16 [T, H, d] tensor whose heads lie side by side."""
    st = t.stride()
    if t.dtype is not _torch.bfloat16 or t.shape != (T, H, d) or st[2] != 1 or (H > 1 and st[1] != d) \
            or t.get_device() != dev:
        raise ValueError(f"{where}: {name} must be a bfloat16 tensor of shape {(T, H, d)} with contiguous heads on "
                         f"cuda:{dev}; got {t.dtype} {tuple(t.shape)} with strides {st} on {t.device}")
    return st[0] if T > 1 else H * d


def _check_norm_rope(where, q, k, q_weight, k_weight, cos, sin, positions, q_out, k_out, of=""):
    """Checks what both directions take (q_out, k_out: the outputs, or, of =
    "d", their gradients): (device, the C call's sizes, token strides of q and k)."""
    torch = _torch or _load_torch()
    dev = _cuda_index(where, q)
    qs, ks, table = q.shape, k.shape, cos.shape
    if len(qs) != 3 or len(ks) != 3 or len(table) != 2:
        raise ValueError(f"{where}: q is [T, H, d], k [T, H_kv, d], cos and sin [max_pos, rot / 2]; got {tuple(qs)}, "
                         f"{tuple(ks)} and {tuple(table)}")
    T, H, d = qs
    H_kv = ks[1]
    sq, sk = _heads_stride(where, "q", q, T, H, d, dev), _heads_stride(where, "k", k, T, H_kv, d, dev)
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    if (q_weight.dtype is not bf16 or q_weight.shape != (d,) or not q_weight.is_contiguous()
            or q_weight.get_device() != dev
            or k_weight.dtype is not bf16 or k_weight.shape != (d,) or not k_weight.is_contiguous()
            or k_weight.get_device() != dev
            or cos.dtype is not f32 or not cos.is_contiguous() or cos.get_device() != dev
            or sin.dtype is not f32 or sin.shape != table or not sin.is_contiguous() or sin.get_device() != dev
            or positions.dtype is not i32 or positions.shape != (T,) or not positions.is_contiguous()
            or positions.get_device() != dev
            or q_out.dtype is not bf16 or q_out.shape != qs or not q_out.is_contiguous() or q_out.get_device() != dev
            or k_out.dtype is not bf16 or k_out.shape != ks or not k_out.is_contiguous()
            or k_out.get_device() != dev):
        _refuse(where, dev, (("q_weight", q_weight, bf16, (d,)), ("k_weight", k_weight, bf16, (d,)),
                             ("cos", cos, f32, table), ("sin", sin, f32, table), ("positions", positions, i32, (T,)),
                             (of + "q_out", q_out, bf16, qs), (of + "k_out", k_out, bf16, ks)))
    return dev, (T, H, H_kv, d, 2 * table[1], table[0], sq, sk)


def fa_qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, q_out, k_out, eps: float = 1e-6,
                    interleaved: bool = False, stream=None) -> None:
    """Per-head norm of q and k with the rotation; same semantics as the C
    entry point. q and k may be strided over tokens (parts of a fused
    projection); the rotated width is 2 * cos.shape[1]."""
    where = "fa_qk_norm_rope"
    dev, sizes = _check_norm_rope(where, q, k, q_weight, k_weight, cos, sin, positions, q_out, k_out)
    st = _on_device(dev, (_LIB or load_library()).fa_qk_norm_rope, q.data_ptr(), k.data_ptr(), q_weight.data_ptr(),
                    k_weight.data_ptr(), cos.data_ptr(), sin.data_ptr(), positions.data_ptr(), q_out.data_ptr(),
                    k_out.data_ptr(), *sizes, float(eps), int(bool(interleaved)), _raw_stream(where, dev, stream))
    if st != FA_OK:
        raise FaError(st, where)


def qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, eps: float = 1e-6, interleaved: bool = False,
                 stream=None):
    """Allocates the outputs [T, H, d] and [T, H_kv, d], then calls fa_qk_norm_rope."""
    torch = _load_torch()
    q_out, k_out = _alloc(stream, lambda: [torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k)])
    fa_qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, q_out, k_out, eps, interleaved, stream)
    return q_out, k_out


def fa_qk_norm_rope_bwd_workspace_size(T: int, H: int, H_kv: int, d: int) -> int:
    return int(load_library().fa_qk_norm_rope_bwd_workspace_size(T, H, H_kv, d))


def fa_qk_norm_rope_bwd(q, k, q_weight, k_weight, cos, sin, positions, dq_out, dk_out, dq, dk, dq_weight, dk_weight,
                        eps: float = 1e-6, interleaved: bool = False, workspace=None, stream=None) -> None:
    """Backward of fa_qk_norm_rope; same semantics as the C entry point. dq
    and dk may be strided over tokens, like q and k."""
    where = "fa_qk_norm_rope_bwd"
    dev, sizes = _check_norm_rope(where, q, k, q_weight, k_weight, cos, sin, positions, dq_out, dk_out, "d")
    T, H, H_kv, d = sizes[:4]
    f32 = _torch.float32
    sq, sk = _heads_stride(where, "dq", dq, T, H, d, dev), _heads_stride(where, "dk", dk, T, H_kv, d, dev)
    if (dq_weight.dtype is not f32 or dq_weight.shape != (d,) or not dq_weight.is_contiguous()
            or dq_weight.get_device() != dev
            or dk_weight.dtype is not f32 or dk_weight.shape != (d,) or not dk_weight.is_contiguous()
            or dk_weight.get_device() != dev):
        _refuse(where, dev, (("dq_weight", dq_weight, f32, (d,)), ("dk_weight", dk_weight, f32, (d,))))
    workspace = _workspace(where, workspace, dev, stream, fa_qk_norm_rope_bwd_workspace_size, T, H, H_kv, d)
    st = _on_device(dev, (_LIB or load_library()).fa_qk_norm_rope_bwd, q.data_ptr(), k.data_ptr(),
                    q_weight.data_ptr(), k_weight.data_ptr(), cos.data_ptr(), sin.data_ptr(), positions.data_ptr(),
                    dq_out.data_ptr(), dk_out.data_ptr(), dq.data_ptr(), dk.data_ptr(), dq_weight.data_ptr(),
                    dk_weight.data_ptr(), *sizes, sq, sk, float(eps), int(bool(interleaved)), workspace.data_ptr(),
                    workspace.numel() * workspace.element_size(), _raw_stream(where, dev, stream))
    if st != FA_OK:
        raise FaError(st, where)


def qk_norm_rope_backward(q, k, q_weight, k_weight, cos, sin, positions, dq_out, dk_out, eps: float = 1e-6,
                          interleaved: bool = False, workspace=None, stream=None):
    """Allocates the gradients, then calls fa_qk_norm_rope_bwd. Returns (dq, dk, dq_weight, dk_weight)."""
    torch = _load_torch()
    dq, dk, dwq, dwk = _alloc(stream, lambda: [
        *(torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k)),
        *(torch.empty(q.shape[2], dtype=torch.float32, device=q.device) for _ in range(2))])
    fa_qk_norm_rope_bwd(q, k, q_weight, k_weight, cos, sin, positions, dq_out, dk_out, dq, dk, dwq, dwk, eps,
                        interleaved, workspace, stream)
    return dq, dk, dwq, dwk


# ---------------------------------------------------------------------------
# The paged cache: tokens appended to it, and the cache held in 4 bits.
# ---------------------------------------------------------------------------
def _check_append(where, q, k, v, cos, sin, positions, slots, q_out):
    """Checks what both forms of the append take besides the cache: (device,
    the C call's pointers up to q_out, its sizes up to max_pos, its strides)."""
    torch = _torch or _load_torch()
    dev = _cuda_index(where, k)
    ks, bf16, i32 = k.shape, torch.bfloat16, torch.int32
    if len(ks) != 3:
        raise ValueError(f"{where}: k and v are [T, H_kv, d], q [T, H, d]; got {tuple(ks)}")
    T, H_kv, d = ks
    kst, vst = k.stride(), v.stride()
    if (k.dtype is not bf16 or v.dtype is not bf16 or v.shape != ks or v.get_device() != dev
            or kst[1:] != (d, 1) or vst[1:] != (d, 1)):
        _heads_stride(where, "k", k, T, H_kv, d, dev)
        _heads_stride(where, "v", v, T, H_kv, d, dev)
    sk, sv = (kst[0], vst[0]) if T > 1 else (H_kv * d, H_kv * d)
    H = sq = qp = qo = None
    if q is not None and q_out is not None:
        qs = q.shape
        if len(qs) != 3:
            raise ValueError(f"{where}: q is [T, H, d]; got {tuple(qs)}")
        H = qs[1]
        sq = _heads_stride(where, "q", q, T, H, d, dev)
        if q_out.dtype is not bf16 or q_out.shape != qs or not q_out.is_contiguous() or q_out.get_device() != dev:
            _refuse(where, dev, (("q_out", q_out, bf16, qs),))
        qp, qo = q.data_ptr(), q_out.data_ptr()
    elif q is not None or q_out is not None:
        raise ValueError(f"{where}: q and q_out go together")
    if slots.dtype is not i32 or slots.shape != (T,) or not slots.is_contiguous() or slots.get_device() != dev:
        _refuse(where, dev, (("slots", slots, i32, (T,)),))
    cp = sp = pp = None
    rot, max_pos = 0, 1
    if cos is not None and sin is not None:
        f32, table = torch.float32, cos.shape
        if len(table) != 2:
            raise ValueError(f"{where}: cos and sin are [max_pos, rot / 2]; got {tuple(table)}")
        if (cos.dtype is not f32 or not cos.is_contiguous() or cos.get_device() != dev
                or sin.dtype is not f32 or sin.shape != table or not sin.is_contiguous() or sin.get_device() != dev):
            _refuse(where, dev, (("cos", cos, f32, table), ("sin", sin, f32, table)))
        max_pos, rot = table[0], 2 * table[1]
        cp, sp = cos.data_ptr(), sin.data_ptr()
    elif cos is not None or sin is not None:
        raise ValueError(f"{where}: cos and sin go together")
    if positions is not None:
        if positions.dtype is not i32 or positions.shape != (T,) or not positions.is_contiguous() \
                or positions.get_device() != dev:
            _refuse(where, dev, (("positions", positions, i32, (T,)),))
        pp = positions.data_ptr()
    elif rot:
        raise ValueError(f"{where}: a rotation needs positions")
    return (dev, (qp, k.data_ptr(), v.data_ptr(), cp, sp, pp, slots.data_ptr(), qo),
            (T, H or 0, H_kv, d, rot, max_pos), (sq or 0, sk, sv))


def fa_kv_append(q, k, v, cos, sin, positions, slots, q_out, k_cache, v_cache, interleaved: bool = False,
                 stream=None) -> None:
    """New tokens rotated and written to a paged cache; same semantics as the
    C entry point. q, k and v may be strided over tokens (parts of a fused
    projection); the rotated width is 2 * cos.shape[1]. q and q_out may both
    be None, and so may cos, sin and positions (no rotation)."""
    where = "fa_kv_append"
    dev, ptrs, sizes, strides = _check_append(where, q, k, v, cos, sin, positions, slots, q_out)
    cs, bf16 = k_cache.shape, _torch.bfloat16
    if len(cs) != 4 or cs[2:] != k.shape[1:]:
        raise ValueError(f"{where}: the caches are [num_blocks, block_size, H_kv, d]; got {tuple(cs)}")
    if (k_cache.dtype is not bf16 or not k_cache.is_contiguous() or k_cache.get_device() != dev
            or v_cache.dtype is not bf16 or v_cache.shape != cs or not v_cache.is_contiguous()
            or v_cache.get_device() != dev):
        _refuse(where, dev, (("k_cache", k_cache, bf16, cs), ("v_cache", v_cache, bf16, cs)))
    args = (*ptrs, k_cache.data_ptr(), v_cache.data_ptr(), *sizes, cs[0], cs[1], *strides, 1 if interleaved else 0,
            _raw_stream(where, dev, stream))
    st = _on_device(dev, (_LIB or load_library()).fa_kv_append, *args)
    if st != FA_OK:
        raise FaError(st, where)


def kv_append(q, k, v, cos, sin, positions, slots, k_cache, v_cache, interleaved: bool = False, stream=None):
    """Allocates the rotated queries [T, H, d], then calls fa_kv_append. Returns
    them (None if q is None)."""
    torch = _load_torch()
    q_out = None if q is None else _alloc(stream, lambda: torch.empty(q.shape, dtype=q.dtype, device=q.device))
    fa_kv_append(q, k, v, cos, sin, positions, slots, q_out, k_cache, v_cache, interleaved, stream)
    return q_out


def _check_q4(where, dev, k_codes, k_scales, v_codes, v_scales, H_kv=None, d=None):
    """Checks the four tensors of a 4-bit cache: (num_blocks, H_kv, block_size, d)."""
    cs, u8, bf16 = k_codes.shape, _torch.uint8, _torch.bfloat16
    if len(cs) != 4 or (d is not None and (cs[1] != H_kv or 2 * cs[3] != d)):
        raise ValueError(f"{where}: the codes are [num_blocks, H_kv, block_size, d / 2]; got {tuple(cs)}")
    ss = (cs[0], cs[1], cs[2], cs[3] // 32, 2)
    if (k_codes.dtype is not u8 or not k_codes.is_contiguous() or k_codes.get_device() != dev
            or v_codes.dtype is not u8 or v_codes.shape != cs or not v_codes.is_contiguous()
            or v_codes.get_device() != dev
            or k_scales.dtype is not bf16 or k_scales.shape != ss or not k_scales.is_contiguous()
            or k_scales.get_device() != dev
            or v_scales.dtype is not bf16 or v_scales.shape != ss or not v_scales.is_contiguous()
            or v_scales.get_device() != dev):
        _refuse(where, dev, (("k_codes", k_codes, u8, cs), ("v_codes", v_codes, u8, cs),
                             ("k_scales", k_scales, bf16, ss), ("v_scales", v_scales, bf16, ss)))
    return cs[0], cs[1], cs[2], 2 * cs[3]


def kv_cache_q4(num_blocks: int, H_kv: int, block_size: int, d: int, device="cuda"):
    """An empty 4-bit cache: (k_codes, k_scales, v_codes, v_scales), all zero."""
    torch = _load_torch()
    shape = (num_blocks, H_kv, block_size)
    return tuple(t for _ in range(2) for t in (
        torch.zeros(*shape, d // 2, dtype=torch.uint8, device=device),
        torch.zeros(*shape, d // 64, 2, dtype=torch.bfloat16, device=device)))


def fa_kv_append_q4(q, k, v, cos, sin, positions, slots, q_out, k_codes, k_scales, v_codes, v_scales,
                    interleaved: bool = False, stream=None) -> None:
    """fa_kv_append for a cache held in 4 bits; same semantics as the C entry point."""
    where = "fa_kv_append_q4"
    dev, ptrs, sizes, strides = _check_append(where, q, k, v, cos, sin, positions, slots, q_out)
    num_blocks, _, block_size, _ = _check_q4(where, dev, k_codes, k_scales, v_codes, v_scales, sizes[2], sizes[3])
    args = (*ptrs, k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(), *sizes,
            num_blocks, block_size, *strides, 1 if interleaved else 0, _raw_stream(where, dev, stream))
    st = _on_device(dev, (_LIB or load_library()).fa_kv_append_q4, *args)
    if st != FA_OK:
        raise FaError(st, where)


def kv_append_q4(q, k, v, cos, sin, positions, slots, k_codes, k_scales, v_codes, v_scales,
                 interleaved: bool = False, stream=None):
    """Allocates the rotated queries [T, H, d], then calls fa_kv_append_q4.
    Returns them (None if q is None)."""
    torch = _load_torch()
    q_out = None if q is None else _alloc(stream, lambda: torch.empty(q.shape, dtype=q.dtype, device=q.device))
    fa_kv_append_q4(q, k, v, cos, sin, positions, slots, q_out, k_codes, k_scales, v_codes, v_scales, interleaved,
                    stream)
    return q_out


def fa_kv_gather_q4(k_codes, k_scales, v_codes, v_scales, block_table, starts, cu_seqlens_k, k, v,
                    stream=None) -> None:
    """Tokens of a 4-bit cache back as packed bf16 keys and values; same
    semantics as the C entry point. starts may be None (token 0)."""
    torch = _torch or _load_torch()
    where = "fa_kv_gather_q4"
    dev = _cuda_index(where, k_codes)
    num_blocks, H_kv, block_size, d = _check_q4(where, dev, k_codes, k_scales, v_codes, v_scales)
    ks, bf16, i32 = k.shape, torch.bfloat16, torch.int32
    if len(ks) != 3 or ks[1] != H_kv or ks[2] != d or block_table.dim() != 2:
        raise ValueError(f"{where}: k and v are [total_k, {H_kv}, {d}], the table [batch, blocks per sequence]; got "
                         f"{tuple(ks)} and {tuple(block_table.shape)}")
    batch, width = block_table.shape
    if (k.dtype is not bf16 or not k.is_contiguous() or k.get_device() != dev
            or v.dtype is not bf16 or v.shape != ks or not v.is_contiguous() or v.get_device() != dev
            or block_table.dtype is not i32 or not block_table.is_contiguous() or block_table.get_device() != dev
            or cu_seqlens_k.dtype is not i32 or cu_seqlens_k.shape != (batch + 1,)
            or not cu_seqlens_k.is_contiguous() or cu_seqlens_k.get_device() != dev):
        _refuse(where, dev, (("k", k, bf16, ks), ("v", v, bf16, ks), ("block_table", block_table, i32, (batch, width)),
                             ("cu_seqlens_k", cu_seqlens_k, i32, (batch + 1,))))
    if starts is not None and (starts.dtype is not i32 or starts.shape != (batch,) or not starts.is_contiguous()
                               or starts.get_device() != dev):
        _refuse(where, dev, (("starts", starts, i32, (batch,)),))
    args = (k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(), block_table.data_ptr(),
            _ptr(starts), cu_seqlens_k.data_ptr(), k.data_ptr(), v.data_ptr(), batch, H_kv, d, ks[0], num_blocks,
            block_size, width, _raw_stream(where, dev, stream))
    st = _on_device(dev, (_LIB or load_library()).fa_kv_gather_q4, *args)
    if st != FA_OK:
        raise FaError(st, where)


def kv_gather_q4(k_codes, k_scales, v_codes, v_scales, block_table, starts, cu_seqlens_k, total_k: int, stream=None):
    """Allocates K and V [total_k, H_kv, d], then calls fa_kv_gather_q4. Returns (K, V)."""
    torch = _load_torch()
    shape = (total_k, k_codes.shape[1], 2 * k_codes.shape[3])
    k, v = _alloc(stream, lambda: [torch.empty(shape, dtype=torch.bfloat16, device=k_codes.device) for _ in range(2)])
    fa_kv_gather_q4(k_codes, k_scales, v_codes, v_scales, block_table, starts, cu_seqlens_k, k, v, stream)
    return k, v


def fa_decode_paged_q4_workspace_size(B: int, n_new: int, H: int, H_kv: int, d: int, max_seq_len: int) -> int:
    return int(load_library().fa_decode_paged_q4_workspace_size(B, n_new, H, H_kv, d, max_seq_len))


def fa_decode_paged_q4(q, k_codes, k_scales, v_codes, v_scales, o, lse, block_table, seq_lens, max_seq_len: int,
                       scale: float, workspace=None, stream=None) -> None:
    """Decoding steps over a 4-bit paged cache with grouped heads; same
    semantics as the C entry point. q and o are [B, n_new, H, d] with lse
    [B, n_new, H], or [B, H, d] and [B, H] for one new query."""
    torch = _torch or _load_torch()
    where = "fa_decode_paged_q4"
    dev = _cuda_index(where, q)
    qs, bf16, i32 = q.shape, torch.bfloat16, torch.int32
    if len(qs) not in (3, 4) or block_table.dim() != 2:
        raise ValueError(f"{where}: q is [B, n_new, H, d] or [B, H, d], the table [B, blocks per sequence]; got "
                         f"{tuple(qs)} and {tuple(block_table.shape)}")
    num_blocks, H_kv, block_size, d = _check_q4(where, dev, k_codes, k_scales, v_codes, v_scales, k_codes.shape[1],
                                                qs[-1])
    B, H = qs[0], qs[-2]
    rows, width = block_table.shape
    if (q.dtype is not bf16 or not q.is_contiguous() or rows != B
            or o.dtype is not bf16 or o.shape != qs or not o.is_contiguous() or o.get_device() != dev
            or lse.dtype is not torch.float32 or lse.shape != qs[:-1] or not lse.is_contiguous()
            or lse.get_device() != dev
            or block_table.dtype is not i32 or not block_table.is_contiguous() or block_table.get_device() != dev
            or seq_lens.dtype is not i32 or seq_lens.shape != (B,) or not seq_lens.is_contiguous()
            or seq_lens.get_device() != dev):
        _refuse(where, dev, (("q", q, bf16, qs), ("o", o, bf16, qs), ("lse", lse, torch.float32, qs[:-1]),
                             ("block_table", block_table, i32, (B, width)), ("seq_lens", seq_lens, i32, (B,))))
    n_new, max_seq_len = qs[1] if len(qs) == 4 else 1, int(max_seq_len)
    workspace = _workspace(where, workspace, dev, stream, fa_decode_paged_q4_workspace_size, B, n_new, H, H_kv, d,
                           max_seq_len)
    args = (q.data_ptr(), k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(),
            o.data_ptr(), lse.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), B, n_new, H, H_kv, d,
            num_blocks, block_size, width, max_seq_len, float(scale), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _raw_stream(where, dev, stream))
    st = _on_device(dev, (_LIB or load_library()).fa_decode_paged_q4, *args)
    if st != FA_OK:
        raise FaError(st, where)


def attention_decode_paged_q4(q, k_codes, k_scales, v_codes, v_scales, block_table, seq_lens, max_seq_len, scale,
                              workspace=None, stream=None):
    """Allocates O and LSE, then calls fa_decode_paged_q4. Returns (O, LSE)."""
    torch = _load_torch()
    o, lse = _alloc(stream, lambda: (torch.empty_like(q),
                                     torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)))
    fa_decode_paged_q4(q, k_codes, k_scales, v_codes, v_scales, o, lse, block_table, seq_lens, max_seq_len, scale,
                       workspace, stream)
    return o, lse


def fa_quantize_fp8(x, out, block_scale, transpose: bool, stream=None) -> None:
    """bf16 [B, H, N, d] -> E4M3 codes (uint8 [B, H, N, d], or [B, H, d, Np]
    with Np = N rounded up to 128 when ``transpose``) and fp32 block scales
    [B, H, ceil(N / 128)]; same semantics as the C entry point."""
    import torch
    _check_bhnd("x", x)
    B, H, N, d = x.shape
    nb = (N + 127) // 128
    shape = (B, H, d, nb * 128) if transpose else (B, H, N, d)
    if out.dtype != torch.uint8 or tuple(out.shape) != shape or not out.is_contiguous():
        raise ValueError(f"out must be contiguous uint8 {shape}")
    if block_scale.dtype != torch.float32 or tuple(block_scale.shape) != (B, H, nb):
        raise ValueError("block_scale must be float32 [B, H, ceil(N / 128)]")
    st = load_library().fa_quantize_fp8(_ptr(x), _ptr(out), _ptr(block_scale), B, H, N, d, int(bool(transpose)),
                                        _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_quantize_fp8")


def quantize_fp8(x, transpose: bool = False, stream=None):
    """Allocates the codes and scales, then calls fa_quantize_fp8."""
    import torch
    B, H, N, d = x.shape
    nb = (N + 127) // 128
    shape = (B, H, d, nb * 128) if transpose else (B, H, N, d)
    out = torch.empty(shape, dtype=torch.uint8, device=x.device)
    sc = torch.empty((B, H, nb), dtype=torch.float32, device=x.device)
    fa_quantize_fp8(x, out, sc, transpose, stream)
    return out, sc


def fa_fwd_fp8(q8, k8, v8t, q_scale, k_scale, v_scale, o, lse, scale: float, causal: bool, kv_lens=None,
               stream=None) -> None:
    """FP8 forward from E4M3 codes and block scales; same semantics as the C entry point."""
    import torch
    B, H, N, d = q8.shape
    nb = (N + 127) // 128
    for name, t, shape in (("q8", q8, (B, H, N, d)), ("k8", k8, (B, H, N, d)), ("v8t", v8t, (B, H, d, nb * 128))):
        if t.dtype != torch.uint8 or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous uint8 {shape}")
    for name, t in (("q_scale", q_scale), ("k_scale", k_scale), ("v_scale", v_scale)):
        if t.dtype != torch.float32 or tuple(t.shape) != (B, H, nb):
            raise ValueError(f"{name} must be float32 [B, H, ceil(N / 128)]")
    _check_bhnd("o", o, (B, H, N, d))
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N):
        raise ValueError("lse must be float32 [B, H, N]")
    st = load_library().fa_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(v8t), _ptr(q_scale), _ptr(k_scale), _ptr(v_scale),
                                   _ptr(o), _ptr(lse), B, H, N, d, float(scale), int(bool(causal)), _ptr(kv_lens),
                                   _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_fwd_fp8")


def attention_forward_fp8(q, k, v, scale: float, causal: bool, kv_lens=None, stream=None):
    """Quantises bf16 Q, K, V (V transposed) and runs the FP8 forward.
    Returns (O, LSE, (q8, q_scale, k8, k_scale, v8t, v_scale))."""
    import torch
    q8, sq = quantize_fp8(q, False, stream)
    k8, sk = quantize_fp8(k, False, stream)
    v8t, sv = quantize_fp8(v, True, stream)
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    fa_fwd_fp8(q8, k8, v8t, sq, sk, sv, o, lse, scale, causal, kv_lens, stream)
    return o, lse, (q8, sq, k8, sk, v8t, sv)


def fa_timing_begin(max_calls: int) -> None:
    st = load_library().fa_timing_begin(int(max_calls))
    if st != FA_OK:
        raise FaError(st, "fa_timing_begin")


def fa_timing_read(kind: int) -> tuple[float, int]:
    """(summed milliseconds, number of timed launches) of one kernel kind."""
    ms = ctypes.c_double(0.0)
    n = ctypes.c_int(0)
    st = load_library().fa_timing_read(int(kind), ctypes.byref(ms), ctypes.byref(n))
    if st != FA_OK:
        raise FaError(st, "fa_timing_read")
    return ms.value, n.value


def fa_timing_end() -> None:
    load_library().fa_timing_end()
