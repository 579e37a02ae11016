"""Exact tiled attention for B200 (sm_100a): thin Python binding of libfa46.so.

Every function here only checks and marshals arguments (device pointers, sizes
and the current CUDA stream) and calls the C ABI declared in include/fa.h; all
arithmetic runs in the library's CUDA kernels.  There is no CPU path: a call
without a CUDA tensor or without the built library raises.

    o, lse = fwd(q, k, v, causal=True)            # prefill forward
    dq, dk, dv = bwd(q, k, v, o, do, lse, causal=True)
    o, lse = decode(q, k_cache, v_cache, seqlens)  # split-KV decode
    o, lse = decode_append(q, k_new, v_new, k_cache, v_cache, seqlens)   # + KV append
    o, lse = decode_paged(q, k_pages, v_pages, page_table, seqlens)     # paged cache

Scores capped by a tanh or biased by distance, documents and prefixes, and a
cache thinned by attention weight:

    o, lse = fwd_scored(q, k, v, causal=True, softcap=50.0, slopes=slopes, docs=doc_ids, prefix=prefix_lens)
    dq, dk, dv = bwd_scored(q, k, v, o, do, lse, causal=True, softcap=50.0, slopes=slopes, docs=doc_ids, prefix=prefix_lens)
    w = key_weights(q, k, lse, causal=True, softcap=50.0)       # attention weight each key receives
    kept = cache_evict(k_cache, v_cache, w, seqlens, keep=1024, recent=128)
    o, lse = decode_scored(q, k_cache, v_cache, seqlens, k_new=k1, v_new=v1, softcap=50.0, weights=w)
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import torch

__all__ = ["fwd", "bwd", "decode", "decode_combine", "device_status", "set_wait_limit_ns",
           "selftest_wait_timeout", "lib", "LIB_PATH", "FA_OK", "FA_ERR_INVALID_ARG",
           "FA_ERR_UNSUPPORTED", "FA_ERR_CUDA", "FA_ERR_TIMEOUT", "FaError",
           "bwd_workspace_size", "decode_workspace_size", "decode_chunk", "launch_guard", "decode_append",
           "decode_paged", "fwd_fp8", "attn_merge", "fwd_scored", "bwd_scored", "decode_scored", "key_weights",
           "cache_evict", "bwd_scored_workspace_size", "scored_workspace_size", "decode_scored_workspace_size",
           "key_weights_workspace_size"]

# FA46_LIBRARY may name another build of the same library (the debug build,
# libfa46_debug.so); there is no fallback when it is missing.
LIB_PATH = os.environ.get("FA46_LIBRARY") or os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfa46.so")
FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT = 0, 1, 2, 3, 4
FA_ERR_DEVICE_INDEX = 5
FA_BF16, FA_FP32 = 0, 1

_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t


class _Score(ctypes.Structure):
    """fa_score"""
    _fields_ = [("softcap", _f), ("slopes", _vp), ("q_docs", _vp), ("k_docs", _vp), ("prefix", _vp)]


class _KvRows(ctypes.Structure):
    """fa_kv_rows"""
    _fields_ = [("k", _vp), ("v", _vp), ("page_table", _vp), ("page_size", _i), ("pages_per_seq", _i),
                ("num_pages", _i)]


_SIGNATURES = {
    "fa_abi_version": ([], _i),
    "fa_debug_build": ([], _i),
    "fa_status_string": ([_i], ctypes.c_char_p),
    "fa_fwd": ([_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp], _i),
    "fa_fwd_ex": ([_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _i, _vp], _i),
    "fa_fwd_fp8": ([_vp, _vp, _vp, _f, _f, _f, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _i, _vp], _i),
    "fa_bwd_workspace_size": ([_i, _i, _i, _i], _sz),
    "fa_bwd": ([_vp] * 9 + [_i] * 6 + [_f, _i, _i, _vp, _sz, _vp], _i),
    "fa_decode_chunk": ([], _i),
    "fa_decode_workspace_size": ([_i, _i, _i, _i], _sz),
    "fa_decode_splitkv": ([_vp] * 6 + [_i] * 5 + [_f, _i, _vp, _sz, _vp], _i),
    "fa_decode_combine": ([_vp] * 5 + [_i] * 5 + [_vp], _i),
    "fa_attn_merge": ([_vp] * 6 + [_i] * 5 + [_vp], _i),
    "fa_decode_append_splitkv": ([_vp] * 8 + [_i] * 5 + [_f, _i, _vp, _sz, _vp], _i),
    "fa_decode_paged_splitkv": ([_vp] * 9 + [_i] * 7 + [_f, _i, _vp, _sz, _vp], _i),
    "fa_decode_splitkv_static": ([_vp] * 6 + [_i] * 5 + [_f, _i, _vp], _i),
    "fa_scored_workspace_size": ([_i, _i, _i], _sz),
    "fa_fwd_scored": ([_vp] * 6 + [_i] * 6 + [_f, _i, ctypes.POINTER(_Score), _i, _vp, _sz, _vp], _i),
    "fa_bwd_scored_workspace_size": ([_i] * 5, _sz),
    "fa_bwd_scored": ([_vp] * 10 + [_i] * 6 + [_f, _i, ctypes.POINTER(_Score), _i, _vp, _sz, _vp], _i),
    "fa_decode_scored_workspace_size": ([_i] * 6, _sz),
    "fa_decode_scored_splitkv": ([_vp] * 11 + [_i] * 8 + [_f, _f, _vp, _i, _vp, _sz, _vp], _i),
    "fa_key_weights_workspace_size": ([_i] * 5, _sz),
    "fa_key_weights": ([_vp] * 4 + [_i] * 8 + [_f, _i, ctypes.POINTER(_Score), _vp, _sz, _vp], _i),
    "fa_cache_evict": ([ctypes.POINTER(_KvRows)] * 2 + [_vp, _i, _vp, _i, _vp, _vp, _vp] + [_i] * 5 + [_vp], _i),
    "fa_device_status": ([ctypes.POINTER(_i), ctypes.POINTER(_i), _i, _vp], _i),
    "fa_set_wait_limit_ns": ([ctypes.c_ulonglong], None),
    "fa_selftest_wait_timeout": ([ctypes.c_ulonglong, _vp], _i),
    "fa_selftest_exp2_poly": ([_vp, _vp, _i, _vp], _i),
    "fa_launch_guard": ([_i, _i, _i, ctypes.POINTER(_i), ctypes.POINTER(_i), ctypes.POINTER(_i)], _i),
}

_lib = None


class FaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {lib().fa_status_string(status).decode()} (status {status})")


def lib() -> ctypes.CDLL:
    """The loaded CUDA library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"CUDA library missing: {LIB_PATH} (run python -m exact_tiled_attention_46_b200.build)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = res
        _lib = handle
    return _lib


def _check(status: int, what: str):
    if status != FA_OK:
        raise FaError(status, what)


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _need(t: torch.Tensor, name: str, dtype=torch.bfloat16, ndim: Optional[int] = None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")


def _odt(dtype) -> int:
    if dtype == torch.bfloat16:
        return FA_BF16
    if dtype == torch.float32:
        return FA_FP32
    raise TypeError("output dtype must be torch.bfloat16 or torch.float32")


def fwd(q, k, v, scale: Optional[float] = None, causal: bool = False, o_dtype=torch.bfloat16,
        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None):
    """Forward attention.  q [B,Lq,Hq,D], k/v [B,Lk,Hkv,D] bf16 -> (o, lse)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, ndim=4)
    B, Lq, Hq, D = q.shape
    _, Lk, Hkv, _ = k.shape
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if out is None:
        out = torch.empty((B, Lq, Hq, D), dtype=o_dtype, device=q.device)
    _need(out, "out", dtype=None, ndim=4)
    if lse is None:
        lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=q.device)
    _need(lse, "lse", dtype=torch.float32, ndim=3)
    _check(lib().fa_fwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                           B, Hq, Hkv, Lq, Lk, D, scale, int(bool(causal)), _odt(out.dtype), _stream(q)),
           "fa_fwd")
    return out, lse


def fwd_fp8(q, k, v, q_scale: float, k_scale: float, v_scale: float, scale: Optional[float] = None,
            causal: bool = False, o_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
            lse: Optional[torch.Tensor] = None):
    """Forward attention on e4m3 inputs (torch.float8_e4m3fn, values = e4m3 * their scale) -> (o, lse)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, dtype=torch.float8_e4m3fn, ndim=4)
    B, Lq, Hq, D = q.shape
    _, Lk, Hkv, _ = k.shape
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if out is None:
        out = torch.empty((B, Lq, Hq, D), dtype=o_dtype, device=q.device)
    _need(out, "out", dtype=None, ndim=4)
    if lse is None:
        lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=q.device)
    _need(lse, "lse", dtype=torch.float32, ndim=3)
    _check(lib().fa_fwd_fp8(q.data_ptr(), k.data_ptr(), v.data_ptr(), float(q_scale), float(k_scale), float(v_scale),
                            out.data_ptr(), lse.data_ptr(), B, Hq, Hkv, Lq, Lk, D, scale, int(bool(causal)),
                            _odt(out.dtype), _stream(q)),
           "fa_fwd_fp8")
    return out, lse


def bwd_workspace_size(B, Hq, Lq, D) -> int:
    return int(lib().fa_bwd_workspace_size(B, Hq, Lq, D))


def bwd(q, k, v, o, do, lse, scale: Optional[float] = None, causal: bool = False, grad_dtype=torch.bfloat16,
        workspace: Optional[torch.Tensor] = None):
    """Backward attention from the saved lse -> (dq, dk, dv)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (do, "do")):
        _need(t, n, ndim=4)
    _need(lse, "lse", dtype=torch.float32, ndim=3)
    B, Lq, Hq, D = q.shape
    _, Lk, Hkv, _ = k.shape
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dq = torch.empty((B, Lq, Hq, D), dtype=grad_dtype, device=q.device)
    dk = torch.empty((B, Lk, Hkv, D), dtype=grad_dtype, device=q.device)
    dv = torch.empty((B, Lk, Hkv, D), dtype=grad_dtype, device=q.device)
    need = bwd_workspace_size(B, Hq, Lq, D)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _check(lib().fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(),
                        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv, Lq, Lk, D, scale,
                        int(bool(causal)), _odt(grad_dtype), workspace.data_ptr(), workspace.numel(), _stream(q)),
           "fa_bwd")
    return dq, dk, dv


def decode_chunk() -> int:
    return int(lib().fa_decode_chunk())


def decode_workspace_size(B, Hq, Lmax, D) -> int:
    return int(lib().fa_decode_workspace_size(B, Hq, Lmax, D))


def decode(q, k_cache, v_cache, seqlens, scale: Optional[float] = None, o_dtype=torch.bfloat16,
           workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
           lse: Optional[torch.Tensor] = None):
    """Split-KV decode.  q [B,Hq,D], caches [B,Lmax,Hkv,D] bf16, seqlens int32 [B] -> (o, lse)."""
    _need(q, "q", ndim=3)
    _need(k_cache, "k_cache", ndim=4)
    _need(v_cache, "v_cache", ndim=4)
    _need(seqlens, "seqlens", dtype=torch.int32, ndim=1)
    B, Hq, D = q.shape
    _, Lmax, Hkv, _ = k_cache.shape
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    need = decode_workspace_size(B, Hq, Lmax, D)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=o_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    _check(lib().fa_decode_splitkv(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), seqlens.data_ptr(),
                                   out.data_ptr(), lse.data_ptr(), B, Hq, Hkv, Lmax, D, scale, _odt(out.dtype),
                                   workspace.data_ptr(), workspace.numel(), _stream(q)),
           "fa_decode_splitkv")
    return out, lse


def decode_append(q, k_new, v_new, k_cache, v_cache, seqlens, scale: Optional[float] = None,
                  o_dtype=torch.bfloat16, workspace: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None):
    """Decode with the new token appended: q [B,Hq,D], k_new/v_new [B,Hkv,D], caches [B,Lmax,Hkv,D].

    Attends over seqlens[b] cached rows plus the new row and writes the new rows
    into the caches at row seqlens[b]; ``seqlens`` is not advanced (add 1 after).
    """
    _need(q, "q", ndim=3)
    _need(k_new, "k_new", ndim=3)
    _need(v_new, "v_new", ndim=3)
    _need(k_cache, "k_cache", ndim=4)
    _need(v_cache, "v_cache", ndim=4)
    _need(seqlens, "seqlens", dtype=torch.int32, ndim=1)
    B, Hq, D = q.shape
    _, Lmax, Hkv, _ = k_cache.shape
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    need = decode_workspace_size(B, Hq, Lmax + 1, D)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=o_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    _check(lib().fa_decode_append_splitkv(q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(),
                                          v_cache.data_ptr(), seqlens.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                          B, Hq, Hkv, Lmax, D, scale, _odt(out.dtype), workspace.data_ptr(),
                                          workspace.numel(), _stream(q)),
           "fa_decode_append_splitkv")
    return out, lse


def decode_paged(q, k_pages, v_pages, page_table, seqlens, k_new=None, v_new=None, scale: Optional[float] = None,
                 o_dtype=torch.bfloat16, workspace: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None):
    """Decode from a paged cache: pages [num_pages,page_size,Hkv,D], page_table int32 [B,pages_per_seq].

    With k_new/v_new [B,Hkv,D] the new token is attended and appended at row
    seqlens[b] (its page must be in the table); ``seqlens`` is not advanced.
    """
    _need(q, "q", ndim=3)
    _need(k_pages, "k_pages", ndim=4)
    _need(v_pages, "v_pages", ndim=4)
    _need(page_table, "page_table", dtype=torch.int32, ndim=2)
    _need(seqlens, "seqlens", dtype=torch.int32, ndim=1)
    append = k_new is not None
    if append:
        _need(k_new, "k_new", ndim=3)
        _need(v_new, "v_new", ndim=3)
    B, Hq, D = q.shape
    num_pages, page_size, Hkv, _ = k_pages.shape
    pages_per_seq = page_table.shape[1]
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    need = decode_workspace_size(B, Hq, pages_per_seq * page_size + int(append), D)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=o_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    _check(lib().fa_decode_paged_splitkv(q.data_ptr(), k_new.data_ptr() if append else None,
                                         v_new.data_ptr() if append else None, k_pages.data_ptr(),
                                         v_pages.data_ptr(), page_table.data_ptr(), seqlens.data_ptr(),
                                         out.data_ptr(), lse.data_ptr(), B, Hq, Hkv, num_pages, page_size,
                                         pages_per_seq, D, scale, _odt(out.dtype), workspace.data_ptr(),
                                         workspace.numel(), _stream(q)),
           "fa_decode_paged_splitkv")
    return out, lse


def decode_combine(o_part, lse_part, num_splits=None, o_dtype=torch.bfloat16):
    """Merge partial results: o_part [B,Hq,S,D], lse_part [B,Hq,S] fp32 -> (o [B,Hq,D], lse [B,Hq])."""
    _need(o_part, "o_part", dtype=torch.float32, ndim=4)
    _need(lse_part, "lse_part", dtype=torch.float32, ndim=3)
    B, Hq, S, D = o_part.shape
    ns_ptr = None
    if num_splits is not None:
        _need(num_splits, "num_splits", dtype=torch.int32, ndim=1)
        ns_ptr = num_splits.data_ptr()
    out = torch.empty((B, Hq, D), dtype=o_dtype, device=o_part.device)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=o_part.device)
    _check(lib().fa_decode_combine(o_part.data_ptr(), lse_part.data_ptr(), ns_ptr, out.data_ptr(), lse.data_ptr(),
                                   B, Hq, D, S, _odt(o_dtype), _stream(o_part)), "fa_decode_combine")
    return out, lse


def attn_merge(o_a, lse_a, o_b, lse_b, out=None, lse_out=None, o_dtype=torch.float32):
    """Merge two results over disjoint key sets: o_* [B,L,H,D] fp32, lse_* [B,H,L] -> (o, lse).

    ``out`` / ``lse_out`` may be ``o_a`` / ``lse_a`` (in-place accumulation).
    """
    _need(o_a, "o_a", dtype=torch.float32, ndim=4)
    _need(o_b, "o_b", dtype=torch.float32, ndim=4)
    _need(lse_a, "lse_a", dtype=torch.float32, ndim=3)
    _need(lse_b, "lse_b", dtype=torch.float32, ndim=3)
    B, L, H, D = o_a.shape
    if out is None:
        out = torch.empty((B, L, H, D), dtype=o_dtype, device=o_a.device)
    _need(out, "out", dtype=None, ndim=4)
    if lse_out is None:
        lse_out = torch.empty((B, H, L), dtype=torch.float32, device=o_a.device)
    _check(lib().fa_attn_merge(o_a.data_ptr(), lse_a.data_ptr(), o_b.data_ptr(), lse_b.data_ptr(), out.data_ptr(),
                               lse_out.data_ptr(), B, H, L, D, _odt(out.dtype), _stream(o_a)), "fa_attn_merge")
    return out, lse_out


# ------------------------------------------------------------ scored attention --
# These calls take a few microseconds on the GPU at small sizes, so their checks
# look at each tensor once and only a tensor that fails is looked at again, for
# the message.
def _shape(t, name: str, shape, dtype, device):
    """t is a contiguous CUDA tensor of this shape, type (None: any) and device."""
    try:
        if (t.shape == shape and (t.dtype is dtype or dtype is None) and t.get_device() == device.index
                and t.is_contiguous()):
            return
    except (AttributeError, RuntimeError):
        pass                                       # not a tensor, or on no device with an index: named below
    _need(t, name, dtype=dtype, ndim=len(shape))
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be on {device}, got {t.device}")


def _space(t, need: int, device):
    """A caller's workspace, checked, or a new one."""
    if t is None:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    _need(t, "workspace", dtype=None)
    if t.device != device:
        raise ValueError(f"workspace must be on {device}, got {t.device}")
    return t


def _bytes(t) -> int:
    return t.numel() * t.element_size()


def _ptr(t):
    return None if t is None else t.data_ptr()


_calls = {}


def _call(device, name: str, *args):
    """One library call on the device's current stream, with that device current."""
    fn = _calls.get(name)
    if fn is None:
        fn = _calls[name] = getattr(lib(), name)
    index = device.index
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch.cuda.current_device() == index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            status = fn(*args, stream)
    if status != FA_OK:
        raise FaError(status, name)


def _qkv(q, k, v=None):
    """(B, Hq, Hkv, Lq, Lk, D) of prefill tensors, checked."""
    _need(q, "q", ndim=4)
    _need(k, "k", ndim=4)
    B, Lq, Hq, D = q.shape
    _, Lk, Hkv, _ = k.shape
    kv, dev = (B, Lk, Hkv, D), q.device
    _shape(k, "k", kv, torch.bfloat16, dev)
    if v is not None:
        _shape(v, "v", kv, torch.bfloat16, dev)
    return B, Hq, Hkv, Lq, Lk, D


def _score(B, Hq, Lq, Lk, device, softcap, slopes, docs, prefix):
    """(fa_score, its tensors).  docs: document numbers [B, L], or a pair for queries [B, Lq] and keys [B, Lk]."""
    qd = kd = None
    if docs is not None:
        qd, kd = docs if isinstance(docs, (tuple, list)) else (docs, docs)
        _shape(qd, "docs of the queries", (B, Lq), torch.int32, device)
        _shape(kd, "docs of the keys", (B, Lk), torch.int32, device)
    if slopes is not None:
        _shape(slopes, "slopes", (Hq,), torch.float32, device)
    if prefix is not None:
        _shape(prefix, "prefix", (B,), torch.int32, device)
    return _Score(float(softcap), _ptr(slopes), _ptr(qd), _ptr(kd), _ptr(prefix))


def scored_workspace_size(B, Lq, Lk) -> int:
    return int(lib().fa_scored_workspace_size(B, Lq, Lk))


def bwd_scored_workspace_size(B, Hq, Lq, Lk, D) -> int:
    return int(lib().fa_bwd_scored_workspace_size(B, Hq, Lq, Lk, D))


def decode_scored_workspace_size(B, Hq, Hkv, rows, D, weights: bool = False) -> int:
    return int(lib().fa_decode_scored_workspace_size(B, Hq, Hkv, rows, D, int(bool(weights))))


def key_weights_workspace_size(B, Hq, Hkv, Lq, Lk) -> int:
    return int(lib().fa_key_weights_workspace_size(B, Hq, Hkv, Lq, Lk))


def fwd_scored(q, k, v, scale: Optional[float] = None, causal: bool = False, softcap: float = 0.0,
               slopes: Optional[torch.Tensor] = None, docs=None, prefix: Optional[torch.Tensor] = None,
               o_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
               o_lo: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Forward attention over capped, biased and masked scores -> (o, lse).

    q [B,Lq,Hq,D], k/v [B,Lk,Hkv,D] bf16.  softcap: scores become softcap *
    tanh(score / softcap) (0: off); slopes fp32 [Hq]: minus slope * distance;
    docs int32 [B,L] or a pair ([B,Lq], [B,Lk]): only pairs of one document
    (negative: none); prefix int32 [B] (causal only): the first keys are seen by
    every query.  o_lo: a bf16 tensor like o that receives what o's rounding took
    off and spares bwd_scored forming O again (o in bf16 only).
    """
    B, Hq, Hkv, Lq, Lk, D = _qkv(q, k, v)
    if o_lo is not None:
        _shape(o_lo, "o_lo", (B, Lq, Hq, D), torch.bfloat16, q.device)
    sc = _score(B, Hq, Lq, Lk, q.device, softcap, slopes, docs, prefix)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dev = q.device
    if out is None:
        out = torch.empty_like(q) if o_dtype is torch.bfloat16 else torch.empty(q.shape, dtype=o_dtype, device=dev)
    else:
        _shape(out, "out", (B, Lq, Hq, D), None, dev)
    if lse is None:
        lse = q.new_empty((B, Hq, Lq), dtype=torch.float32)
    else:
        _shape(lse, "lse", (B, Hq, Lq), torch.float32, dev)
    ws = _space(workspace, scored_workspace_size(B, Lq, Lk), dev) if docs is not None else None
    _call(dev, "fa_fwd_scored", q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), _ptr(o_lo), lse.data_ptr(),
          B, Hq, Hkv, Lq, Lk, D, scale, int(bool(causal)), ctypes.byref(sc), _odt(out.dtype), _ptr(ws),
          0 if ws is None else _bytes(ws))
    return out, lse


def bwd_scored(q, k, v, o, do, lse, scale: Optional[float] = None, causal: bool = False, softcap: float = 0.0,
               slopes: Optional[torch.Tensor] = None, docs=None, prefix: Optional[torch.Tensor] = None,
               grad_dtype=torch.bfloat16, o_lo: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None):
    """Backward of fwd_scored (same score arguments) from its o, o_lo and lse -> (dq, dk, dv).

    Without o_lo the call forms O again, to 16 bits, which takes a forward's time.
    """
    B, Hq, Hkv, Lq, Lk, D = _qkv(q, k, v)
    if o_lo is not None:
        _shape(o_lo, "o_lo", q.shape, torch.bfloat16, q.device)
    _shape(o, "o", q.shape, torch.bfloat16, q.device)
    _shape(do, "do", q.shape, torch.bfloat16, q.device)
    _shape(lse, "lse", (B, Hq, Lq), torch.float32, q.device)
    sc = _score(B, Hq, Lq, Lk, q.device, softcap, slopes, docs, prefix)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dt, dev = _odt(grad_dtype), q.device
    dq, dk, dv = (torch.empty_like(t, dtype=grad_dtype) for t in (q, k, v))
    ws = _space(workspace, bwd_scored_workspace_size(B, Hq, Lq, Lk, D), dev)
    _call(dev, "fa_bwd_scored", q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _ptr(o_lo), do.data_ptr(),
          lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv, Lq, Lk, D, scale, int(bool(causal)),
          ctypes.byref(sc), dt, ws.data_ptr(), _bytes(ws))
    return dq, dk, dv


def _cache(k, v, page_table, B, D, device):
    """(Hkv, num_pages, page_size, pages_per_seq) of a contiguous or paged cache, checked."""
    shape = num, rows, Hkv, _ = k.shape
    _shape(k, "k_cache", (num, rows, Hkv, D), torch.bfloat16, device)
    _shape(v, "v_cache", shape, torch.bfloat16, device)
    if page_table is None:
        if num != B:
            raise ValueError(f"k_cache must hold {B} sequences, got {num}")
        return Hkv, num, rows, 1
    pages = page_table.shape[-1]
    _shape(page_table, "page_table", (B, pages), torch.int32, device)
    return Hkv, num, rows, pages


def _weights(w, B, Hkv, device):
    """Row length of accumulated weights [B, Hkv, rows], checked."""
    ld = w.shape[-1] if isinstance(w, torch.Tensor) else 0
    _shape(w, "weights", (B, Hkv, ld), torch.float32, device)
    return ld


def decode_scored(q, k_cache, v_cache, seqlens, page_table: Optional[torch.Tensor] = None, k_new=None, v_new=None,
                  scale: Optional[float] = None, softcap: float = 0.0, slopes: Optional[torch.Tensor] = None,
                  starts: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None,
                  o_dtype=torch.bfloat16, workspace: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None):
    """One new token over capped and biased scores: q [B,Hq,D] -> (o, lse).

    Cache [B,Lmax,Hkv,D], or pages [num_pages,page_size,Hkv,D] with page_table
    int32 [B,pages_per_seq].  k_new/v_new [B,Hkv,D] are attended and written at
    row seqlens[b] (``seqlens`` is not advanced).  starts int32 [B]: first row
    attended.  weights fp32 [B,Hkv,>= rows]: every attended row's attention
    weight, summed over the kv head's query heads, is added in place (set for
    the appended row).
    """
    _need(q, "q", ndim=3)
    _need(k_cache, "k_cache", ndim=4)
    B, Hq, D = q.shape
    dev = q.device
    Hkv, num, page, pps = _cache(k_cache, v_cache, page_table, B, D, dev)
    _shape(seqlens, "seqlens", (B,), torch.int32, dev)
    append = k_new is not None or v_new is not None
    if append:
        if k_new is None or v_new is None:
            raise ValueError("k_new and v_new come together")
        _shape(k_new, "k_new", (B, Hkv, D), torch.bfloat16, dev)
        _shape(v_new, "v_new", (B, Hkv, D), torch.bfloat16, dev)
    if slopes is not None:
        _shape(slopes, "slopes", (Hq,), torch.float32, dev)
    if starts is not None:
        _shape(starts, "starts", (B,), torch.int32, dev)
    ld = 0 if weights is None else _weights(weights, B, Hkv, dev)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q) if o_dtype is torch.bfloat16 else torch.empty(q.shape, dtype=o_dtype, device=dev)
    else:
        _shape(out, "out", (B, Hq, D), None, dev)
    if lse is None:
        lse = q.new_empty((B, Hq), dtype=torch.float32)
    else:
        _shape(lse, "lse", (B, Hq), torch.float32, dev)
    ws = _space(workspace, decode_scored_workspace_size(B, Hq, Hkv, page * pps + int(append), D, weights is not None),
                dev)
    _call(dev, "fa_decode_scored_splitkv", q.data_ptr(), _ptr(k_new), _ptr(v_new), k_cache.data_ptr(),
          v_cache.data_ptr(), _ptr(page_table), seqlens.data_ptr(), _ptr(starts), out.data_ptr(), lse.data_ptr(),
          _ptr(weights), ld, B, Hq, Hkv, num, page, pps, D, scale, float(softcap), _ptr(slopes), _odt(out.dtype),
          ws.data_ptr(), _bytes(ws))
    return out, lse


def key_weights(q, k, lse, scale: Optional[float] = None, causal: bool = False, softcap: float = 0.0,
                slopes: Optional[torch.Tensor] = None, docs=None, prefix: Optional[torch.Tensor] = None,
                weights: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Attention weight each key receives from q's queries, summed over them and the kv head's query heads.

    q [B,Lq,Hq,D], k [B,Lk,Hkv,D] bf16, lse [B,Hq,Lq] and the score arguments as
    in fwd_scored.  Returns fp32 [B,Hkv,Lk]; with ``weights`` [B,Hkv,>= Lk] the
    sums are added to its first Lk columns instead.
    """
    B, Hq, Hkv, Lq, Lk, D = _qkv(q, k)
    _shape(lse, "lse", (B, Hq, Lq), torch.float32, q.device)
    sc = _score(B, Hq, Lq, Lk, q.device, softcap, slopes, docs, prefix)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    add = weights is not None
    if add:
        _weights(weights, B, Hkv, q.device)
    else:
        weights = torch.empty((B, Hkv, Lk), dtype=torch.float32, device=q.device)
    ws = _space(workspace, key_weights_workspace_size(B, Hq, Hkv, Lq, Lk), q.device)
    _call(q.device, "fa_key_weights", q.data_ptr(), k.data_ptr(), lse.data_ptr(), weights.data_ptr(),
          weights.shape[2], int(add), B, Hq, Hkv, Lq, Lk, D, scale, int(bool(causal)), ctypes.byref(sc), ws.data_ptr(),
          _bytes(ws))
    return weights


def cache_evict(k_cache, v_cache, weights, seqlens, keep: int, recent: int = 0,
                page_table: Optional[torch.Tensor] = None, out=None, kept: Optional[torch.Tensor] = None):
    """Keep the ``recent`` last rows of each sequence and its keep - recent heaviest others, per kv head -> kept.

    Cache as in decode_scored, weights fp32 [B,Hkv,>= rows], seqlens int32 [B].
    The kept rows move in order to the cache's first rows, with their weights,
    and seqlens becomes min(seqlens, keep), all in place; or into ``out`` =
    (k, v, weights, seqlens) or (k, v, weights, seqlens, page_table), which
    overlaps none of the inputs.  Sequences of at most ``keep`` rows are kept
    whole.  kept int32 [B,Hkv,keep]: the rows they came from, -1 past the end.
    """
    _need(k_cache, "k_cache", ndim=4)
    B, D, dev = len(seqlens), k_cache.shape[3], k_cache.device
    _shape(seqlens, "seqlens", (B,), torch.int32, dev)
    Hkv, num, page, pps = _cache(k_cache, v_cache, page_table, B, D, dev)
    ld = _weights(weights, B, Hkv, dev)
    src = dst = _KvRows(k_cache.data_ptr(), v_cache.data_ptr(), _ptr(page_table), page, pps, num)
    w2, n2, ld2 = weights, seqlens, ld
    if out is not None:
        k2, v2, w2, n2 = out[:4]
        table2 = out[4] if len(out) > 4 else None
        _need(k2, "out k", ndim=4)
        _shape(n2, "out seqlens", (B,), torch.int32, dev)
        Hkv2, num, page, pps = _cache(k2, v2, table2, B, D, dev)
        if Hkv2 != Hkv:
            raise ValueError(f"out must hold {Hkv} kv heads, got {Hkv2}")
        ld2 = _weights(w2, B, Hkv, dev)
        dst = _KvRows(k2.data_ptr(), v2.data_ptr(), _ptr(table2), page, pps, num)
    if kept is None:
        kept = seqlens.new_empty((B, Hkv, max(int(keep), 0)))
    else:
        _shape(kept, "kept", (B, Hkv, int(keep)), torch.int32, dev)
    _call(dev, "fa_cache_evict", ctypes.byref(src), ctypes.byref(dst), weights.data_ptr(), ld, w2.data_ptr(), ld2,
          seqlens.data_ptr(), n2.data_ptr(), kept.data_ptr(), B, Hkv, D, int(keep),
          int(recent))
    return kept


def device_status(reset: bool = False, device=None):
    """(code, where) of the library's device status word (synchronises)."""
    code, where = ctypes.c_int(0), ctypes.c_int(0)
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    st = torch.cuda.current_stream(dev).cuda_stream
    _check(lib().fa_device_status(ctypes.byref(code), ctypes.byref(where), int(reset), st), "fa_device_status")
    return code.value, where.value


def set_wait_limit_ns(ns: int):
    lib().fa_set_wait_limit_ns(int(ns))


def selftest_wait_timeout(wait_ns: int, device=None):
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    _check(lib().fa_selftest_wait_timeout(int(wait_ns), torch.cuda.current_stream(dev).cuda_stream),
           "fa_selftest_wait_timeout")


def launch_guard(bwd: bool, D: int, causal: bool, query_regs: bool = True):
    """(compiled registers or None, registers the split assumes, cached check result) of one kernel instantiation."""
    regs, exp, state = ctypes.c_int(-1), ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().fa_launch_guard(int(bool(bwd)), int(D), int(bool(causal)),
                                 ctypes.byref(regs) if query_regs else None, ctypes.byref(exp), ctypes.byref(state)),
           "fa_launch_guard")
    return (regs.value if query_regs else None), exp.value, state.value
