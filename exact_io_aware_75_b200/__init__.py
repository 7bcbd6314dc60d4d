"""Exact IO-aware attention for B200 (sm_100a): Python binding of libfa_sm100.so.

The binding only marshals arguments: it takes torch CUDA tensors, passes their
device pointers, sizes and the current CUDA stream to the C ABI declared in
``include/fa.h``, and raises :class:`FAError` on a non-zero status.  All
arithmetic runs in the library's kernels.  There is no fallback: if the
shared library is missing or fails to load, importing this package raises.
With ``stream=s`` a call runs inside ``torch.cuda.stream(s)``, what it allocates
included; a stream of another device than the tensors' is refused.

Functions mirror the C entry points:
    fwd            -> fa_fwd            (dense prefill)
    fwd_varlen     -> fa_fwd_varlen     (packed sequences, cu_seqlens)
    bwd            -> fa_bwd            (dense backward: dQ, dK, dV)
    bwd_varlen     -> fa_bwd_varlen     (packed-sequence backward)
    decode_paged   -> fa_decode_paged   (paged split-KV decode)
    fp8_prepare    -> fa_fp8_prepare    (Hadamard rotation + E4M3 operands)
    fwd_fp8        -> fa_fwd_fp8        (FP8 prefill on those operands)
    fwd_cross, fwd_varlen_cross, bwd_cross, bwd_varlen_cross
                   -> fa_*_cross        (cross attention and its backward)
    decode_shared  -> fa_decode_shared  (paged decode with shared prefixes)
    decode_cross   -> fa_decode_cross   (few queries against encoder states)
    cache_fork, cache_append, cache_copy_pages, cache_collect, cache_compact
                   -> fa_cache_*        (the pages of the cache)
    decode_paged_noalloc, decode_workspace_bytes, bwd_workspace_bytes,
    check_device_error, selftest_watchdog, status_string, version
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa_sm100.so")

FA_OK = 0
FA_ERR_INVALID_ARG = -1
FA_ERR_UNSUPPORTED = -2
FA_ERR_ALIGNMENT = -3
FA_ERR_WORKSPACE = -4
FA_ERR_CUDA = -5
FA_ERR_TIMEOUT = -6
FA_ERR_PAGES = -7
FA_OUT_BF16 = 0
FA_OUT_FP32 = 1

EXPORTS = ("fa_fwd", "fa_fwd_varlen", "fa_fwd_sinks", "fa_fwd_varlen_sinks", "fa_fwd_paged",
           "fa_fwd_doc", "fa_fwd_sink_tokens", "fa_fwd_varlen_sink_tokens",
           "fa_bwd_workspace_bytes", "fa_bwd", "fa_bwd_varlen", "fa_bwd_sinks",
           "fa_bwd_varlen_sinks",
           "fa_decode_workspace_bytes", "fa_decode_paged", "fa_decode_paged_sinks",
           "fa_decode_paged_fp8", "fa_fp8_workspace_bytes", "fa_fp8_prepare", "fa_fwd_fp8",
           "fa_fwd_cross", "fa_fwd_varlen_cross", "fa_bwd_cross", "fa_bwd_varlen_cross",
           "fa_decode_shared_workspace_bytes", "fa_decode_shared",
           "fa_decode_cross_workspace_bytes", "fa_decode_cross",
           "fa_cache_fork", "fa_cache_append", "fa_cache_copy_pages",
           "fa_cache_collect_workspace_bytes", "fa_cache_collect",
           "fa_cache_compact_workspace_bytes", "fa_cache_compact",
           "fa_decode_paged_noalloc", "fa_status_string", "fa_check_device_error",
           "fa_selftest_watchdog", "fa_version")


class FAError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} (status {status})")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing; build it with `python exact_io_aware_75_b200/build.py` "
            "(or __graft_entry__.build()).  There is no fallback path.")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp] + [i] * 7 + [f, i, vp]
    lib.fa_fwd.restype = i
    lib.fa_fwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp] + [i] * 8 + [f, i, vp]
    lib.fa_fwd_varlen.restype = i
    lib.fa_fwd_sinks.argtypes = [vp] * 6 + [i] * 7 + [f, i, vp]
    lib.fa_fwd_sinks.restype = i
    lib.fa_fwd_varlen_sinks.argtypes = [vp] * 7 + [i] * 8 + [f, i, vp]
    lib.fa_fwd_varlen_sinks.restype = i
    lib.fa_decode_paged_sinks.argtypes = [vp] * 8 + [i] * 7 + [f, vp, sz, vp]
    lib.fa_decode_paged_sinks.restype = i
    lib.fa_fwd_sink_tokens.argtypes = [vp] * 5 + [i] * 7 + [f, i, vp]
    lib.fa_fwd_sink_tokens.restype = i
    lib.fa_fwd_varlen_sink_tokens.argtypes = [vp] * 6 + [i] * 8 + [f, i, vp]
    lib.fa_fwd_varlen_sink_tokens.restype = i
    lib.fa_fwd_doc.argtypes = [vp] * 6 + [i] * 7 + [f, i, vp]
    lib.fa_fwd_doc.restype = i
    lib.fa_fwd_paged.argtypes = [vp] * 9 + [i] * 11 + [f, i, vp]
    lib.fa_fwd_paged.restype = i
    lib.fa_decode_paged_fp8.argtypes = [vp] * 10 + [i] * 7 + [f, vp, sz, vp]
    lib.fa_decode_paged_fp8.restype = i
    lib.fa_fp8_workspace_bytes.argtypes = [i] * 3
    lib.fa_fp8_workspace_bytes.restype = sz
    lib.fa_fp8_prepare.argtypes = [vp] * 10 + [i] * 5 + [vp, sz, vp]
    lib.fa_fp8_prepare.restype = i
    lib.fa_fwd_fp8.argtypes = [vp] * 8 + [i] * 7 + [f, i, vp]
    lib.fa_fwd_fp8.restype = i
    lib.fa_bwd_workspace_bytes.argtypes = [i] * 3
    lib.fa_bwd_workspace_bytes.restype = sz
    lib.fa_bwd.argtypes = [vp] * 9 + [i] * 7 + [f, vp, sz, vp]
    lib.fa_bwd.restype = i
    lib.fa_bwd_varlen.argtypes = [vp] * 10 + [i] * 8 + [f, vp, sz, vp]
    lib.fa_bwd_varlen.restype = i
    lib.fa_bwd_sinks.argtypes = [vp] * 11 + [i] * 7 + [f, vp, sz, vp]
    lib.fa_bwd_sinks.restype = i
    lib.fa_bwd_varlen_sinks.argtypes = [vp] * 12 + [i] * 8 + [f, vp, sz, vp]
    lib.fa_bwd_varlen_sinks.restype = i
    lib.fa_decode_workspace_bytes.argtypes = [i] * 5
    lib.fa_decode_workspace_bytes.restype = sz
    lib.fa_decode_paged.argtypes = [vp] * 7 + [i] * 7 + [f, vp, sz, vp]
    lib.fa_decode_paged.restype = i
    lib.fa_decode_paged_noalloc.argtypes = [vp] * 7 + [i] * 7 + [f, vp]
    lib.fa_decode_paged_noalloc.restype = i
    lib.fa_fwd_cross.argtypes = [vp] * 6 + [i] * 6 + [f, i, vp]
    lib.fa_fwd_cross.restype = i
    lib.fa_fwd_varlen_cross.argtypes = [vp] * 7 + [i] * 8 + [f, i, vp]
    lib.fa_fwd_varlen_cross.restype = i
    lib.fa_bwd_cross.argtypes = [vp] * 10 + [i] * 6 + [f, vp, sz, vp]
    lib.fa_bwd_cross.restype = i
    lib.fa_bwd_varlen_cross.argtypes = [vp] * 11 + [i] * 8 + [f, vp, sz, vp]
    lib.fa_bwd_varlen_cross.restype = i
    lib.fa_decode_shared_workspace_bytes.argtypes = [i] * 4
    lib.fa_decode_shared_workspace_bytes.restype = sz
    lib.fa_decode_shared.argtypes = [vp] * 10 + [i] * 8 + [f, vp, sz, vp]
    lib.fa_decode_shared.restype = i
    lib.fa_decode_cross_workspace_bytes.argtypes = [i] * 5
    lib.fa_decode_cross_workspace_bytes.restype = sz
    lib.fa_decode_cross.argtypes = [vp] * 6 + [i] * 6 + [f, vp, sz, vp]
    lib.fa_decode_cross.restype = i
    lib.fa_cache_fork.argtypes = ([vp] * 4 + [i, vp, vp, i, vp, i, vp, vp, i] + [vp] * 3 + [i] * 5
                                  + [vp])
    lib.fa_cache_fork.restype = i
    lib.fa_cache_append.argtypes = ([vp] * 3 + [i, i] + [vp] * 6 + [i, vp, vp] + [i] * 5 + [vp])
    lib.fa_cache_append.restype = i
    lib.fa_cache_copy_pages.argtypes = [vp] * 4 + [i, vp, vp] + [i] * 5 + [vp]
    lib.fa_cache_copy_pages.restype = i
    lib.fa_cache_collect_workspace_bytes.argtypes = [i]
    lib.fa_cache_collect_workspace_bytes.restype = sz
    lib.fa_cache_collect.argtypes = [vp] * 2 + [i] * 4 + [vp] * 3 + [sz, vp]
    lib.fa_cache_collect.restype = i
    lib.fa_cache_compact_workspace_bytes.argtypes = [i]
    lib.fa_cache_compact_workspace_bytes.restype = sz
    lib.fa_cache_compact.argtypes = [vp] * 4 + [i, vp, vp, i] + [vp] * 3 + [i] * 5 + [vp, sz, vp]
    lib.fa_cache_compact.restype = i
    lib.fa_status_string.argtypes = [i]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_check_device_error.argtypes = [vp]
    lib.fa_check_device_error.restype = i
    lib.fa_selftest_watchdog.argtypes = [vp]
    lib.fa_selftest_watchdog.restype = i
    lib.fa_version.argtypes = []
    lib.fa_version.restype = i
    return lib


_lib = _load()


def library():
    """The loaded ctypes handle (for tests that call the C ABI directly)."""
    return _lib


def status_string(status: int) -> str:
    return _lib.fa_status_string(int(status)).decode()


def version() -> int:
    return int(_lib.fa_version())


# The argument checks run on every call, next to kernels of a few microseconds:
# plain integers for pointers, the raw stream handle, no objects made in passing.
def _ptr(t):
    return t.data_ptr() if t is not None else None


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _inside(f, stream, args):
    """f(..., stream=s) as f(...) inside torch.cuda.stream(s), so that what f allocates (its
    workspace, outputs not passed) belongs to s: in the pool of the caller's stream a
    workspace could be handed out again while the kernels on s still use it.  ``args``: f's
    arguments by name.  (A line in each call instead of a decorator, which cost every call
    without a stream 0.5 us.)"""
    name, x = next(iter(args.items()))
    if isinstance(x, dict):                  # fp8_prepare's operands
        x = next(iter(x.values()), None)
    if isinstance(x, torch.Tensor) and x.is_cuda and x.device != stream.device:
        raise FAError(FA_ERR_INVALID_ARG, f"a stream of {stream.device}, {name} on {x.device}")
    args["stream"] = None
    with torch.cuda.stream(stream):
        return f(**args)


def _check(rc: int, where: str):
    if rc != FA_OK:
        raise FAError(rc, where)


_Tensor, _int32 = torch.Tensor, torch.int32


def _need(t, dtype, ndim, name):
    if (isinstance(t, _Tensor) and t.dtype is dtype and t.dim() == ndim and t.is_cuda
            and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise FAError(FA_ERR_INVALID_ARG, f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise FAError(FA_ERR_INVALID_ARG, f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise FAError(FA_ERR_INVALID_ARG, f"{name} must have {ndim} dims, got {t.dim()}")
    if not t.is_contiguous():
        raise FAError(FA_ERR_INVALID_ARG, f"{name} must be contiguous")


def fwd(q, k, v, causal=False, window=0, scale=None, out_dtype=torch.bfloat16,
        out=None, lse=None, return_lse=True, stream=None, sinks=None, doc_ids=None,
        sink_tokens=None):
    """Dense prefill.  q [B,N,Hq,d], k/v [B,N,Hkv,d] bf16 -> (O [B,N,Hq,d], LSE [B,Hq,N]).
    ``sinks`` (fp32 [Hq], device) selects fa_fwd_sinks; ``doc_ids`` (int32 [B,N],
    device) selects fa_fwd_doc; ``sink_tokens`` (an int, with causal and a window)
    selects fa_fwd_sink_tokens."""
    if stream is not None:
        return _inside(fwd, stream, locals())
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, torch.bfloat16, 4, n)
    B, N, Hq, d = q.shape
    Hkv = k.shape[2]
    if tuple(k.shape) != (B, N, Hkv, d) or tuple(v.shape) != (B, N, Hkv, d):
        raise FAError(FA_ERR_INVALID_ARG, "k/v shape")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, N, Hq, d), dtype=out_dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    od = FA_OUT_FP32 if out.dtype == torch.float32 else FA_OUT_BF16
    if sink_tokens is not None:
        if sinks is not None or doc_ids is not None or not causal:
            raise FAError(FA_ERR_UNSUPPORTED, "sink_tokens with sinks, doc_ids or non-causal")
        _check(_lib.fa_fwd_sink_tokens(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq,
                                       Hkv, N, d, int(window), int(sink_tokens), float(scale),
                                       od, _stream(stream)), "fa_fwd_sink_tokens")
        return out, lse
    if doc_ids is not None:
        if sinks is not None:
            raise FAError(FA_ERR_UNSUPPORTED, "sinks with doc_ids")
        _need(doc_ids, torch.int32, 2, "doc_ids")
        if tuple(doc_ids.shape) != (B, N):
            raise FAError(FA_ERR_INVALID_ARG, "doc_ids shape")
        _check(_lib.fa_fwd_doc(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(doc_ids),
                               B, Hq, Hkv, N, d, int(causal), int(window), float(scale), od,
                               _stream(stream)), "fa_fwd_doc")
        return out, lse
    if sinks is not None:
        _need(sinks, torch.float32, 1, "sinks")
        _check(_lib.fa_fwd_sinks(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(sinks),
                                 B, Hq, Hkv, N, d, int(causal), int(window), float(scale), od,
                                 _stream(stream)), "fa_fwd_sinks")
        return out, lse
    _check(_lib.fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, N, d,
                       int(causal), int(window), float(scale), od, _stream(stream)), "fa_fwd")
    return out, lse


FP8_BLOCK = 128   # tokens per Q / K scale block


def fp8_workspace_bytes(B, N, Hkv) -> int:
    return int(_lib.fa_fp8_workspace_bytes(int(B), int(N), int(Hkv)))


def fp8_prepare(q, k, v, signs=None, out=None, workspace=None, stream=None):
    """E4M3 operands of the FP8 prefill.  q [B,N,Hq,128], k/v [B,N,Hkv,128] bf16;
    signs fp32 [128] of +-1 (device) or None (no rotation).  Returns a dict with
    q8 [B,N,Hq,128], k8 [B,N,Hkv,128] uint8 codes, vt8 [B,Hkv,128,vt_stride]
    uint8 (V transposed), q_scale [B,Hq,nblk], k_scale [B,Hkv,nblk], v_scale
    [B,Hkv] fp32.  ``out`` may be such a dict to fill in place."""
    if stream is not None:
        return _inside(fp8_prepare, stream, locals())
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, torch.bfloat16, 4, n)
    B, N, Hq, d = q.shape
    Hkv = k.shape[2]
    if tuple(k.shape) != (B, N, Hkv, d) or tuple(v.shape) != (B, N, Hkv, d):
        raise FAError(FA_ERR_INVALID_ARG, "k/v shape")
    if signs is not None:
        _need(signs, torch.float32, 1, "signs")
        if signs.numel() != d:
            raise FAError(FA_ERR_INVALID_ARG, "signs shape")
    nblk = (N + FP8_BLOCK - 1) // FP8_BLOCK
    vts = (N + 15) // 16 * 16
    dev = q.device
    if out is None:
        out = {"q8": torch.empty((B, N, Hq, d), dtype=torch.uint8, device=dev),
               "k8": torch.empty((B, N, Hkv, d), dtype=torch.uint8, device=dev),
               "vt8": torch.empty((B, Hkv, d, vts), dtype=torch.uint8, device=dev),
               "q_scale": torch.empty((B, Hq, nblk), dtype=torch.float32, device=dev),
               "k_scale": torch.empty((B, Hkv, nblk), dtype=torch.float32, device=dev),
               "v_scale": torch.empty((B, Hkv), dtype=torch.float32, device=dev)}
    ws_need = fp8_workspace_bytes(B, N, Hkv)
    if workspace is None:
        workspace = torch.empty(max(ws_need, 4), dtype=torch.uint8, device=dev)
    _check(_lib.fa_fp8_prepare(_ptr(q), _ptr(k), _ptr(v), _ptr(signs), _ptr(out["q8"]),
                               _ptr(out["k8"]), _ptr(out["vt8"]), _ptr(out["q_scale"]),
                               _ptr(out["k_scale"]), _ptr(out["v_scale"]), B, N, Hq, Hkv, d,
                               _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _stream(stream)), "fa_fp8_prepare")
    return out


def fwd_fp8(prep, causal=False, window=0, scale=None, out_dtype=torch.bfloat16, out=None,
            lse=None, return_lse=True, stream=None):
    """FP8 prefill on fp8_prepare's operands -> (O [B,N,Hq,128], LSE [B,Hq,N])."""
    if stream is not None:
        return _inside(fwd_fp8, stream, locals())
    q8, k8, vt8 = prep["q8"], prep["k8"], prep["vt8"]
    _need(q8, torch.uint8, 4, "q8")
    _need(k8, torch.uint8, 4, "k8")
    _need(vt8, torch.uint8, 4, "vt8")
    B, N, Hq, d = q8.shape
    Hkv = k8.shape[2]
    if tuple(k8.shape) != (B, N, Hkv, d) or tuple(vt8.shape) != (B, Hkv, d, (N + 15) // 16 * 16):
        raise FAError(FA_ERR_INVALID_ARG, "k8/vt8 shape")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, N, Hq, d), dtype=out_dtype, device=q8.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q8.device)
    od = FA_OUT_FP32 if out.dtype == torch.float32 else FA_OUT_BF16
    _check(_lib.fa_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(vt8), _ptr(prep["q_scale"]),
                           _ptr(prep["k_scale"]), _ptr(prep["v_scale"]), _ptr(out), _ptr(lse),
                           B, Hq, Hkv, N, d, int(causal), int(window), float(scale), od,
                           _stream(stream)), "fa_fwd_fp8")
    return out, lse


def fwd_varlen(q, k, v, cu_seqlens, max_seqlen, causal=False, window=0, scale=None,
               out_dtype=torch.bfloat16, out=None, lse=None, return_lse=True, stream=None,
               sinks=None, sink_tokens=None):
    """Packed prefill.  q [T,Hq,d], k/v [T,Hkv,d], cu_seqlens [S+1] int32 (device)
    -> (O [T,Hq,d], LSE [Hq,T]).  ``sinks`` selects fa_fwd_varlen_sinks;
    ``sink_tokens`` (an int, with causal and a window) fa_fwd_varlen_sink_tokens."""
    if stream is not None:
        return _inside(fwd_varlen, stream, locals())
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, torch.bfloat16, 3, n)
    _need(cu_seqlens, torch.int32, 1, "cu_seqlens")
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((T, Hq, d), dtype=out_dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
    od = FA_OUT_FP32 if out.dtype == torch.float32 else FA_OUT_BF16
    if sink_tokens is not None:
        if sinks is not None or not causal:
            raise FAError(FA_ERR_UNSUPPORTED, "sink_tokens with sinks or non-causal")
        _check(_lib.fa_fwd_varlen_sink_tokens(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                              _ptr(cu_seqlens), cu_seqlens.numel() - 1, T,
                                              int(max_seqlen), Hq, Hkv, d, int(window),
                                              int(sink_tokens), float(scale), od,
                                              _stream(stream)), "fa_fwd_varlen_sink_tokens")
        return out, lse
    if sinks is not None:
        _need(sinks, torch.float32, 1, "sinks")
        _check(_lib.fa_fwd_varlen_sinks(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                        _ptr(sinks), _ptr(cu_seqlens), cu_seqlens.numel() - 1,
                                        T, int(max_seqlen), Hq, Hkv, d, int(causal),
                                        int(window), float(scale), od, _stream(stream)),
               "fa_fwd_varlen_sinks")
        return out, lse
    _check(_lib.fa_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                              _ptr(cu_seqlens), cu_seqlens.numel() - 1, T, int(max_seqlen),
                              Hq, Hkv, d, int(causal), int(window), float(scale), od,
                              _stream(stream)), "fa_fwd_varlen")
    return out, lse


def fwd_paged(q, k_cache, v_cache, block_table, cu_seqlens_q, seq_lens_k, max_seqlen_q,
              causal=True, window=0, scale=None, sinks=None, out_dtype=torch.bfloat16, out=None,
              lse=None, return_lse=True, stream=None):
    """Chunked prefill over a paged cache.  q [Tq,Hq,d] (each sequence's last L_q
    tokens), caches [P,16,Hkv,d], block_table [S,maxp], cu_seqlens_q [S+1],
    seq_lens_k [S] -> (O [Tq,Hq,d], LSE [Hq,Tq])."""
    if stream is not None:
        return _inside(fwd_paged, stream, locals())
    _need(q, torch.bfloat16, 3, "q")
    _need(k_cache, torch.bfloat16, 4, "k_cache")
    _need(v_cache, torch.bfloat16, 4, "v_cache")
    _need(block_table, torch.int32, 2, "block_table")
    _need(cu_seqlens_q, torch.int32, 1, "cu_seqlens_q")
    _need(seq_lens_k, torch.int32, 1, "seq_lens_k")
    T, Hq, d = q.shape
    P, ps, Hkv, _ = k_cache.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((T, Hq, d), dtype=out_dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
    if sinks is not None:
        _need(sinks, torch.float32, 1, "sinks")
    od = FA_OUT_FP32 if out.dtype == torch.float32 else FA_OUT_BF16
    _check(_lib.fa_fwd_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                             _ptr(cu_seqlens_q), _ptr(seq_lens_k), _ptr(out), _ptr(lse),
                             _ptr(sinks), cu_seqlens_q.numel() - 1, T, int(max_seqlen_q), P,
                             Hq, Hkv, d, ps, block_table.shape[1], int(causal), int(window),
                             float(scale), od, _stream(stream)), "fa_fwd_paged")
    return out, lse


def bwd_workspace_bytes(total_tokens, Hq, d) -> int:
    return int(_lib.fa_bwd_workspace_bytes(int(total_tokens), int(Hq), int(d)))


def bwd(q, k, v, o, dout, lse, causal=False, window=0, scale=None, dq=None, dk=None, dv=None,
        workspace=None, stream=None, sinks=None, dsinks=None):
    """Dense backward.  q/o/dout [B,N,Hq,d], k/v [B,N,Hkv,d] bf16, lse [B,Hq,N] fp32
    (from fwd) -> (dQ, dK, dV) bf16; with ``sinks`` (the forward's sink logits,
    fp32 [Hq]) fa_bwd_sinks, returning (dQ, dK, dV, dsinks)."""
    if stream is not None:
        return _inside(bwd, stream, locals())
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        _need(t, torch.bfloat16, 4, n)
    _need(lse, torch.float32, 3, "lse")
    B, N, Hq, d = q.shape
    Hkv = k.shape[2]
    if (tuple(k.shape) != (B, N, Hkv, d) or tuple(v.shape) != (B, N, Hkv, d)
            or tuple(o.shape) != (B, N, Hq, d) or tuple(dout.shape) != (B, N, Hq, d)
            or tuple(lse.shape) != (B, Hq, N)):
        raise FAError(FA_ERR_INVALID_ARG, "bwd shapes")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if workspace is None:
        workspace = torch.empty(max(bwd_workspace_bytes(B * N, Hq, d), 1), dtype=torch.uint8,
                                device=q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if sinks is not None:
        _need(sinks, torch.float32, 1, "sinks")
        if dsinks is None:
            dsinks = torch.empty((Hq,), dtype=torch.float32, device=q.device)
        _check(_lib.fa_bwd_sinks(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                                 _ptr(sinks), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dsinks), B, Hq,
                                 Hkv, N, d, int(causal), int(window), float(scale),
                                 _ptr(workspace), workspace.numel(), _stream(stream)),
               "fa_bwd_sinks")
        return dq, dk, dv, dsinks
    _check(_lib.fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq),
                       _ptr(dk), _ptr(dv), B, Hq, Hkv, N, d, int(causal), int(window),
                       float(scale), _ptr(workspace), workspace.numel(), _stream(stream)),
           "fa_bwd")
    return dq, dk, dv


def bwd_varlen(q, k, v, o, dout, lse, cu_seqlens, max_seqlen, causal=False, window=0,
               scale=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Packed backward.  q/o/dout [T,Hq,d], k/v [T,Hkv,d], lse [Hq,T], cu_seqlens [S+1]
    -> (dQ, dK, dV) bf16."""
    if stream is not None:
        return _inside(bwd_varlen, stream, locals())
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        _need(t, torch.bfloat16, 3, n)
    _need(lse, torch.float32, 2, "lse")
    _need(cu_seqlens, torch.int32, 1, "cu_seqlens")
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if workspace is None:
        workspace = torch.empty(max(bwd_workspace_bytes(T, Hq, d), 1), dtype=torch.uint8,
                                device=q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check(_lib.fa_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                              _ptr(dq), _ptr(dk), _ptr(dv), _ptr(cu_seqlens),
                              cu_seqlens.numel() - 1, T, int(max_seqlen), Hq, Hkv, d,
                              int(causal), int(window), float(scale), _ptr(workspace),
                              workspace.numel(), _stream(stream)), "fa_bwd_varlen")
    return dq, dk, dv


def _out_pair(out, lse, o_shape, lse_shape, out_dtype, return_lse, like):
    """The output tensors of a forward call: given ones checked, missing ones made on
    like's device."""
    if out is None:
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise FAError(FA_ERR_INVALID_ARG, f"out_dtype {out_dtype}")
        out = (torch.empty_like(like) if like.dtype is out_dtype and like.shape == o_shape
               else like.new_empty(o_shape, dtype=out_dtype))
    else:
        _need(out, torch.float32 if out.dtype == torch.float32 else torch.bfloat16, len(o_shape), "out")
        if out.shape != o_shape:
            raise FAError(FA_ERR_INVALID_ARG, "out shape")
    if lse is not None:
        _need(lse, torch.float32, len(lse_shape), "lse")
        if lse.shape != lse_shape:
            raise FAError(FA_ERR_INVALID_ARG, "lse shape")
    elif return_lse:
        lse = like.new_empty(lse_shape, dtype=torch.float32)
    return out, lse, FA_OUT_FP32 if out.dtype == torch.float32 else FA_OUT_BF16


def _decode_out(out, lse, o_shape, lse_shape, return_lse, like):
    """As _out_pair, for calls whose O is bf16."""
    if out is not None and getattr(out, "dtype", None) != torch.bfloat16:
        raise FAError(FA_ERR_INVALID_ARG, "out must be torch.bfloat16")
    return _out_pair(out, lse, o_shape, lse_shape, torch.bfloat16, return_lse, like)[:2]


def _same(t, ref, name):
    """A tensor of ref's type and shape."""
    _need(t, ref.dtype, ref.dim(), name)
    if t.shape != ref.shape:
        raise FAError(FA_ERR_INVALID_ARG, f"{name} shape")
    return t


def _like(t, ref, name):
    return torch.empty_like(ref) if t is None else _same(t, ref, name)


@functools.lru_cache(maxsize=None)
def _sm_count(device):
    return torch.cuda.get_device_properties(device).multi_processor_count


def _split_is_faster(B, Nq, Nk, Hq, Hkv, d, sms):
    """Whether fa_decode_cross takes less than fa_fwd_cross, by estimates in us of both.

    fa_fwd_cross: 256 rows (a KV head's query heads of some tokens) to an SM, a block of 128
    keys 2.1 us, 1.75 for up to 128 rows.  fa_decode_cross: the blocks spread over all SMs,
    1.35 us each at d = 128 and 0.8 to 1.1 at 64, 2.2 for more than 128 rows; a start and a
    join that grow with the rows.  Over 90 sizes (1 to 150 queries, 300 and 3,000 keys, B 1 to
    12, 8/1, 16/16 and 32/8 heads) the worse one was taken at most 5 us beside the better."""
    group = Hq // Hkv
    tokens = 128 // group if group <= 128 else 128
    heads = Hkv if group <= 128 else Hq
    rows, blocks = Nq * group, -(-Nk // 128)
    waves = -(-B * heads * -(-Nq // (2 * tokens)) // sms)
    whole = 8 + waves * blocks * (2.1 if Nq > tokens else 1.75)
    pairs = -(-rows // 256)
    each = 2.2 if rows > 128 else 1.35 if d == 128 else 0.8 if rows <= 16 else 1.1
    start = 10 if rows <= 8 else 13 if rows <= 32 else 19
    return start + B * Hkv * pairs * blocks * each / sms + B * Nq * Hq * 1e-3 < whole


def _cross_shapes(q, k, v, ndim):
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, torch.bfloat16, ndim, n)
    if v.shape != k.shape or k.shape[-1] != q.shape[-1] or (ndim == 4 and k.shape[0] != q.shape[0]):
        raise FAError(FA_ERR_INVALID_ARG, "q/k/v shape")


def fwd_cross(q, k, v, seq_lens_k=None, scale=None, out_dtype=torch.bfloat16, out=None, lse=None,
              return_lse=True, stream=None, split_keys=None):
    """Cross attention, dense.  q [B,Nq,Hq,d], k/v [B,Nk,Hkv,d] bf16, seq_lens_k [B] int32
    (device) or None -> (O [B,Nq,Hq,d], LSE [B,Hq,Nq]).  split_keys: through
    decode_cross (bf16 O only), or not; by default where the queries are few, as include/fa.h
    says there."""
    if stream is not None:
        return _inside(fwd_cross, stream, locals())
    _cross_shapes(q, k, v, 4)
    B, Nq, Hq, d = q.shape
    Nk, Hkv = k.shape[1:3]
    if seq_lens_k is not None:
        _need_ints((B,), "seq_lens_k", seq_lens_k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, lse, od = _out_pair(out, lse, (B, Nq, Hq, d), (B, Hq, Nq), out_dtype, return_lse, q)
    if split_keys is None:
        split_keys = (od == FA_OUT_BF16 and 0 < Hkv <= Hq and Hq % Hkv == 0 and Nk < 1 << 22
                      and _split_is_faster(B, Nq, Nk, Hq, Hkv, d, _sm_count(q.get_device()))
                      and decode_cross_workspace_bytes(B, Hq, Hkv, Nq, d) > 0)
    if split_keys:
        return decode_cross(q, k, v, seq_lens_k, scale, out, lse, return_lse=False, stream=stream)
    with _device_of(q, k, v, seq_lens_k, out, lse):
        _check(_lib.fa_fwd_cross(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(seq_lens_k),
                                 B, Hq, Hkv, Nq, Nk, d, float(scale), od, _stream(stream)),
               "fa_fwd_cross")
    return out, lse


def fwd_varlen_cross(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale=None,
                     out_dtype=torch.bfloat16, out=None, lse=None, return_lse=True, stream=None):
    """Cross attention, packed.  q [Tq,Hq,d], k/v [Tk,Hkv,d] bf16, cu_seqlens_q and
    cu_seqlens_k [S+1] int32 (device) -> (O [Tq,Hq,d], LSE [Hq,Tq])."""
    if stream is not None:
        return _inside(fwd_varlen_cross, stream, locals())
    _cross_shapes(q, k, v, 3)
    Tq, Hq, d = q.shape
    Tk, Hkv = k.shape[:2]
    _need(cu_seqlens_q, torch.int32, 1, "cu_seqlens_q")
    _need_ints(cu_seqlens_q.shape, "cu_seqlens_k", cu_seqlens_k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, lse, od = _out_pair(out, lse, (Tq, Hq, d), (Hq, Tq), out_dtype, return_lse, q)
    with _device_of(q, k, v, cu_seqlens_q, cu_seqlens_k, out,
                    lse):
        _check(_lib.fa_fwd_varlen_cross(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                        _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
                                        cu_seqlens_q.numel() - 1, Tq, Tk, int(max_seqlen_q),
                                        int(max_seqlen_k), Hq, Hkv, d, float(scale), od,
                                        _stream(stream)), "fa_fwd_varlen_cross")
    return out, lse


def bwd_cross(q, k, v, o, dout, lse, seq_lens_k=None, scale=None, dq=None, dk=None, dv=None,
              workspace=None, stream=None):
    """Backward of fwd_cross.  q/o/dout [B,Nq,Hq,d], k/v [B,Nk,Hkv,d] bf16, lse [B,Hq,Nq]
    -> (dQ, dK, dV) bf16."""
    if stream is not None:
        return _inside(bwd_cross, stream, locals())
    _cross_shapes(q, k, v, 4)
    B, Nq, Hq, d = q.shape
    Nk, Hkv = k.shape[1:3]
    _same(o, q, "o")
    _same(dout, q, "dout")
    _need(lse, torch.float32, 3, "lse")
    if tuple(lse.shape) != (B, Hq, Nq):
        raise FAError(FA_ERR_INVALID_ARG, "lse shape")
    if seq_lens_k is not None:
        _need_ints((B,), "seq_lens_k", seq_lens_k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq, dk, dv = _like(dq, q, "dq"), _like(dk, k, "dk"), _like(dv, v, "dv")
    workspace = _bytes_of(workspace, bwd_workspace_bytes(B * Nq, Hq, d), q)
    with _device_of(q, k, v, o, dout, lse, seq_lens_k, dq, dk,
                    dv, workspace):
        _check(_lib.fa_bwd_cross(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                                 _ptr(dq), _ptr(dk), _ptr(dv), _ptr(seq_lens_k), B, Hq, Hkv, Nq,
                                 Nk, d, float(scale), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream)),
               "fa_bwd_cross")
    return dq, dk, dv


def bwd_varlen_cross(q, k, v, o, dout, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
                     scale=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Backward of fwd_varlen_cross.  q/o/dout [Tq,Hq,d], k/v [Tk,Hkv,d] bf16, lse [Hq,Tq]
    -> (dQ, dK, dV) bf16."""
    if stream is not None:
        return _inside(bwd_varlen_cross, stream, locals())
    _cross_shapes(q, k, v, 3)
    Tq, Hq, d = q.shape
    Tk, Hkv = k.shape[:2]
    _same(o, q, "o")
    _same(dout, q, "dout")
    _need(lse, torch.float32, 2, "lse")
    if tuple(lse.shape) != (Hq, Tq):
        raise FAError(FA_ERR_INVALID_ARG, "lse shape")
    _need(cu_seqlens_q, torch.int32, 1, "cu_seqlens_q")
    _need_ints(cu_seqlens_q.shape, "cu_seqlens_k", cu_seqlens_k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq, dk, dv = _like(dq, q, "dq"), _like(dk, k, "dk"), _like(dv, v, "dv")
    workspace = _bytes_of(workspace, bwd_workspace_bytes(Tq, Hq, d), q)
    with _device_of(q, k, v, o, dout, lse, cu_seqlens_q,
                    cu_seqlens_k, dq, dk, dv, workspace):
        _check(_lib.fa_bwd_varlen_cross(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                                        _ptr(dq), _ptr(dk), _ptr(dv), _ptr(cu_seqlens_q),
                                        _ptr(cu_seqlens_k), cu_seqlens_q.numel() - 1, Tq, Tk,
                                        int(max_seqlen_q), int(max_seqlen_k), Hq, Hkv, d,
                                        float(scale), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(),
                                        _stream(stream)), "fa_bwd_varlen_cross")
    return dq, dk, dv


def decode_shared_workspace_bytes(num_seqs, Hq, Hkv, d) -> int:
    return int(_lib.fa_decode_shared_workspace_bytes(int(num_seqs), int(Hq), int(Hkv), int(d)))


def decode_shared(q, k_cache, v_cache, block_table, seq_lens, cu_groups, prefix_lens, scale=None,
                  sinks=None, out=None, lse=None, return_lse=True, workspace=None, stream=None):
    """Paged decode of sequences that share prefixes.  q [S,Hq,d], caches [P,16,Hkv,d],
    block_table [S,maxp], seq_lens [S], cu_groups [G+1], prefix_lens [G] int32: the sequences
    of group g name the same pages for their first prefix_lens[g] // 16 table entries
    -> (O [S,Hq,d] bf16, LSE [S,Hq])."""
    if stream is not None:
        return _inside(decode_shared, stream, locals())
    _need(q, torch.bfloat16, 3, "q")
    _need(k_cache, torch.bfloat16, 4, "k_cache")
    _need(v_cache, torch.bfloat16, 4, "v_cache")
    _need(block_table, torch.int32, 2, "block_table")
    S, Hq, d = q.shape
    P, ps, Hkv, dk = k_cache.shape
    maxp = block_table.shape[1]
    if v_cache.shape != k_cache.shape or dk != d or block_table.shape[0] != S:
        raise FAError(FA_ERR_INVALID_ARG, "shapes")
    _need_ints((S,), "seq_lens", seq_lens)
    _need(prefix_lens, torch.int32, 1, "prefix_lens")
    groups = prefix_lens.shape[0]
    _need_ints((groups + 1,), "cu_groups", cu_groups)
    if sinks is not None:
        _need(sinks, torch.float32, 1, "sinks")
        if sinks.shape[0] != Hq:
            raise FAError(FA_ERR_INVALID_ARG, "sinks shape")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, lse = _decode_out(out, lse, (S, Hq, d), (S, Hq), return_lse, q)
    workspace = _bytes_of(workspace, decode_shared_workspace_bytes(S, Hq, max(Hkv, 1), d), q)
    with _device_of(q, k_cache, v_cache, block_table,
                    seq_lens, cu_groups, prefix_lens, sinks,
                    out, lse, workspace):
        _check(_lib.fa_decode_shared(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                     _ptr(seq_lens), _ptr(cu_groups), _ptr(prefix_lens),
                                     _ptr(out), _ptr(lse), _ptr(sinks), S, groups, P, Hq, Hkv, d,
                                     ps, maxp, float(scale), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(),
                                     _stream(stream)), "fa_decode_shared")
    return out, lse


def decode_cross_workspace_bytes(B, Hq, Hkv, Nq, d) -> int:
    return int(_lib.fa_decode_cross_workspace_bytes(int(B), int(Hq), int(Hkv), int(Nq), int(d)))


def decode_cross(q, k, v, seq_lens_k=None, scale=None, out=None, lse=None, return_lse=True,
                 workspace=None, stream=None):
    """Cross attention of few queries, the keys split over the GPU.  q [B,Nq,Hq,d], k/v
    [B,Nk,Hkv,d] bf16, seq_lens_k [B] int32 (device) or None -> (O [B,Nq,Hq,d] bf16,
    LSE [B,Hq,Nq])."""
    if stream is not None:
        return _inside(decode_cross, stream, locals())
    _cross_shapes(q, k, v, 4)
    B, Nq, Hq, d = q.shape
    Nk, Hkv = k.shape[1:3]
    if seq_lens_k is not None:
        _need_ints((B,), "seq_lens_k", seq_lens_k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, lse = _decode_out(out, lse, (B, Nq, Hq, d), (B, Hq, Nq), return_lse, q)
    workspace = _bytes_of(workspace, decode_cross_workspace_bytes(B, Hq, max(Hkv, 1), Nq, d), q)
    with _device_of(q, k, v, seq_lens_k, out, lse, workspace):
        _check(_lib.fa_decode_cross(_ptr(q), _ptr(k), _ptr(v), _ptr(seq_lens_k), _ptr(out),
                                    _ptr(lse), B, Hq, Hkv, Nq, Nk, d, float(scale),
                                    _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _stream(stream)), "fa_decode_cross")
    return out, lse


def decode_workspace_bytes(num_seqs, Hq, d, page_size, max_pages_per_seq) -> int:
    return int(_lib.fa_decode_workspace_bytes(int(num_seqs), int(Hq), int(d), int(page_size),
                                              int(max_pages_per_seq)))


def decode_paged(q, k_cache, v_cache, block_table, seq_lens, scale=None, out=None, lse=None,
                 return_lse=True, workspace=None, stream=None, sinks=None):
    """Paged decode.  q [S,Hq,d], caches [P,ps,Hkv,d], block_table [S,maxp] int32,
    seq_lens [S] int32 -> (O [S,Hq,d] bf16, LSE [S,Hq])."""
    if stream is not None:
        return _inside(decode_paged, stream, locals())
    _need(q, torch.bfloat16, 3, "q")
    _need(k_cache, torch.bfloat16, 4, "k_cache")
    _need(v_cache, torch.bfloat16, 4, "v_cache")
    _need(block_table, torch.int32, 2, "block_table")
    _need(seq_lens, torch.int32, 1, "seq_lens")
    S, Hq, d = q.shape
    P, ps, Hkv, _ = k_cache.shape
    maxp = block_table.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    need = decode_workspace_bytes(S, Hq, d, ps, maxp)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty((S, Hq, d), dtype=torch.bfloat16, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((S, Hq), dtype=torch.float32, device=q.device)
    if sinks is not None:
        _need(sinks, torch.float32, 1, "sinks")
        _check(_lib.fa_decode_paged_sinks(_ptr(q), _ptr(k_cache), _ptr(v_cache),
                                          _ptr(block_table), _ptr(seq_lens), _ptr(out),
                                          _ptr(lse), _ptr(sinks), S, P, Hq, Hkv, d, ps, maxp,
                                          float(scale), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(),
                                          _stream(stream)), "fa_decode_paged_sinks")
        return out, lse
    _check(_lib.fa_decode_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                _ptr(seq_lens), _ptr(out), _ptr(lse), S, P, Hq, Hkv, d, ps,
                                maxp, float(scale), _ptr(workspace),
                                workspace.numel() * workspace.element_size(),
                                _stream(stream)), "fa_decode_paged")
    return out, lse


def decode_paged_fp8(q, k_codes, v_codes, k_scale, v_scale, block_table, seq_lens, scale=None,
                     sinks=None, out=None, lse=None, return_lse=True, workspace=None,
                     stream=None):
    """Paged decode over an FP8 E4M3 cache.  k_codes/v_codes [P,ps,Hkv,d] uint8 (or
    float8_e4m3fn), k_scale/v_scale [P,Hkv] fp32 -> (O [S,Hq,d] bf16, LSE [S,Hq])."""
    if stream is not None:
        return _inside(decode_paged_fp8, stream, locals())
    _need(q, torch.bfloat16, 3, "q")
    if k_codes.dtype == torch.float8_e4m3fn:
        k_codes, v_codes = k_codes.view(torch.uint8), v_codes.view(torch.uint8)
    _need(k_codes, torch.uint8, 4, "k_codes")
    _need(v_codes, torch.uint8, 4, "v_codes")
    _need(k_scale, torch.float32, 2, "k_scale")
    _need(v_scale, torch.float32, 2, "v_scale")
    _need(block_table, torch.int32, 2, "block_table")
    _need(seq_lens, torch.int32, 1, "seq_lens")
    S, Hq, d = q.shape
    P, ps, Hkv, _ = k_codes.shape
    maxp = block_table.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    need = decode_workspace_bytes(S, Hq, d, ps, maxp)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty((S, Hq, d), dtype=torch.bfloat16, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((S, Hq), dtype=torch.float32, device=q.device)
    if sinks is not None:
        _need(sinks, torch.float32, 1, "sinks")
    _check(_lib.fa_decode_paged_fp8(_ptr(q), _ptr(k_codes), _ptr(v_codes), _ptr(k_scale),
                                    _ptr(v_scale), _ptr(block_table), _ptr(seq_lens), _ptr(out),
                                    _ptr(lse), _ptr(sinks), S, P, Hq, Hkv, d, ps, maxp,
                                    float(scale), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(),
                                    _stream(stream)), "fa_decode_paged_fp8")
    return out, lse


def decode_paged_noalloc(q, k_cache, v_cache, block_table, seq_lens, scale=None, out=None,
                         lse=None, return_lse=True, stream=None):
    """Paged decode with the library's fixed device scratch instead of a
    workspace, for callers that cannot allocate device memory (see
    fa_decode_paged_noalloc in include/fa.h: 32 MiB limit, first call per
    device before any stream capture, overlapping calls race)."""
    if stream is not None:
        return _inside(decode_paged_noalloc, stream, locals())
    _need(q, torch.bfloat16, 3, "q")
    _need(k_cache, torch.bfloat16, 4, "k_cache")
    _need(v_cache, torch.bfloat16, 4, "v_cache")
    _need(block_table, torch.int32, 2, "block_table")
    _need(seq_lens, torch.int32, 1, "seq_lens")
    S, Hq, d = q.shape
    P, ps, Hkv, _ = k_cache.shape
    maxp = block_table.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((S, Hq, d), dtype=torch.bfloat16, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((S, Hq), dtype=torch.float32, device=q.device)
    _check(_lib.fa_decode_paged_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache),
                                        _ptr(block_table), _ptr(seq_lens), _ptr(out),
                                        _ptr(lse), S, P, Hq, Hkv, d, ps, maxp, float(scale),
                                        _stream(stream)), "fa_decode_paged_noalloc")
    return out, lse


_same_device = contextlib.nullcontext()


def _device_of(first, *others):
    """A context in which the device of `first` is current; the others must be on it."""
    device = first.get_device()
    for t in others:
        if t is not None and t.get_device() != device:
            raise FAError(FA_ERR_INVALID_ARG, f"a tensor on {t.device}, others on {first.device}")
    return _same_device if device == torch.cuda.current_device() else torch.cuda.device(device)


def _need_cache(k_cache, v_cache, k_scale, v_scale):
    """Checks a paged cache and its scales; returns it with E4M3 values as uint8
    codes, and the bytes of an element."""
    if isinstance(k_cache, torch.Tensor) and k_cache.dtype == torch.float8_e4m3fn:
        k_cache = k_cache.view(torch.uint8)
    if isinstance(v_cache, torch.Tensor) and v_cache.dtype == torch.float8_e4m3fn:
        v_cache = v_cache.view(torch.uint8)
    dtype = k_cache.dtype if getattr(k_cache, "dtype", None) == torch.uint8 else torch.bfloat16
    _need(k_cache, dtype, 4, "k_cache")
    _need(v_cache, dtype, 4, "v_cache")
    if v_cache.shape != k_cache.shape:
        raise FAError(FA_ERR_INVALID_ARG, "v_cache shape")
    if dtype == torch.uint8:
        _need(k_scale, torch.float32, 2, "k_scale")
        _need(v_scale, torch.float32, 2, "v_scale")
        want = (k_cache.shape[0], k_cache.shape[2])
        if tuple(k_scale.shape) != want or tuple(v_scale.shape) != want:
            raise FAError(FA_ERR_INVALID_ARG, "k_scale/v_scale shape")
    elif k_scale is not None or v_scale is not None:
        raise FAError(FA_ERR_INVALID_ARG, "scales with a bf16 cache")
    return k_cache, v_cache, 1 if dtype == torch.uint8 else 2


def _need_ints(shape, name, t):
    if (isinstance(t, _Tensor) and t.dtype is _int32 and t.shape == shape and t.is_cuda
            and t.is_contiguous()):
        return
    _need(t, _int32, len(shape), name)
    if t.shape != shape:
        raise FAError(FA_ERR_INVALID_ARG, f"{name} shape {tuple(t.shape)}, not {tuple(shape)}")


def _bytes_of(workspace, need, like):
    if workspace is None:
        return like.new_empty(max(need, 1), dtype=torch.uint8)
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
        raise FAError(FA_ERR_WORKSPACE, "workspace must be a contiguous CUDA tensor")
    return workspace


def cache_fork(k_cache, v_cache, block_table, seq_lens, parents, free_pages, free_count,
               block_table_out, seq_lens_out, free_count_out, k_scale=None, v_scale=None,
               stream=None):
    """The next batch of slots: slot i continues slot parents[i] (-1: empty), sharing full
    pages and copying a partly filled last page for all but the first that continue it.
    caches [P,16,Hkv,d] (bf16, or E4M3 with scales [P,Hkv]), block_table [S,maxp], seq_lens
    [S], parents [N], free_pages [F], free_count [1] int32 -> writes block_table_out [N,maxp],
    seq_lens_out [N], free_count_out [1], which must not overlap the inputs."""
    if stream is not None:
        return _inside(cache_fork, stream, locals())
    k_cache, v_cache, eb = _need_cache(k_cache, v_cache, k_scale, v_scale)
    P, ps, Hkv, d = k_cache.shape
    _need(block_table, torch.int32, 2, "block_table")
    _need(parents, torch.int32, 1, "parents")
    S, maxp = block_table.shape
    N = parents.shape[0]
    _need_ints((S,), "seq_lens", seq_lens)
    _need(free_pages, torch.int32, 1, "free_pages")
    _need_ints((1,), "free_count", free_count)
    _need_ints((N, maxp), "block_table_out", block_table_out)
    _need_ints((N,), "seq_lens_out", seq_lens_out)
    _need_ints((1,), "free_count_out", free_count_out)
    with _device_of(k_cache, v_cache, k_scale, v_scale,
                    block_table, seq_lens, parents,
                    free_pages, free_count, block_table_out,
                    seq_lens_out, free_count_out):
        _check(_lib.fa_cache_fork(_ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), eb,
                                  _ptr(block_table), _ptr(seq_lens), S, _ptr(parents), N,
                                  _ptr(free_pages), _ptr(free_count), free_pages.shape[0],
                                  _ptr(block_table_out), _ptr(seq_lens_out),
                                  _ptr(free_count_out), P, Hkv, d, ps, maxp,
                                  _stream(stream)), "fa_cache_fork")


def cache_append(k_new, v_new, cu_new, k_cache, v_cache, block_table, seq_lens, free_pages,
                 free_count, seq_lens_out, free_count_out, stream=None):
    """New tokens behind the sequences' ends.  k_new, v_new [T,Hkv,d] bf16 packed by cu_new
    [S+1]; caches [P,16,Hkv,d] bf16; block_table [S,maxp] (gets the pages taken), seq_lens
    [S], free_pages [F], free_count [1] int32 -> writes seq_lens_out [S], free_count_out [1],
    which must not be the inputs."""
    if stream is not None:
        return _inside(cache_append, stream, locals())
    _need(k_new, torch.bfloat16, 3, "k_new")
    _need(v_new, torch.bfloat16, 3, "v_new")
    _need(k_cache, torch.bfloat16, 4, "k_cache")
    _need(v_cache, torch.bfloat16, 4, "v_cache")
    P, ps, Hkv, d = k_cache.shape
    T = k_new.shape[0]
    if v_cache.shape != k_cache.shape or tuple(k_new.shape) != (T, Hkv, d) or v_new.shape != k_new.shape:
        raise FAError(FA_ERR_INVALID_ARG, "k_new/v_new/v_cache shape")
    _need(block_table, torch.int32, 2, "block_table")
    S, maxp = block_table.shape
    _need_ints((S + 1,), "cu_new", cu_new)
    _need_ints((S,), "seq_lens", seq_lens)
    _need(free_pages, torch.int32, 1, "free_pages")
    _need_ints((1,), "free_count", free_count)
    _need_ints((S,), "seq_lens_out", seq_lens_out)
    _need_ints((1,), "free_count_out", free_count_out)
    with _device_of(k_cache, v_cache, k_new, v_new, cu_new,
                    block_table, seq_lens, free_pages,
                    free_count, seq_lens_out,
                    free_count_out):
        _check(_lib.fa_cache_append(_ptr(k_new), _ptr(v_new), _ptr(cu_new), S, T, _ptr(k_cache),
                                    _ptr(v_cache), _ptr(block_table), _ptr(seq_lens),
                                    _ptr(free_pages), _ptr(free_count), free_pages.shape[0],
                                    _ptr(seq_lens_out), _ptr(free_count_out), P, Hkv, d, ps, maxp, _stream(stream)),
               "fa_cache_append")


def cache_copy_pages(k_cache, v_cache, src, dst, k_scale=None, v_scale=None, stream=None):
    """Page src[i] of the caches to page dst[i] (int32 [n], device), with its scales."""
    if stream is not None:
        return _inside(cache_copy_pages, stream, locals())
    k_cache, v_cache, eb = _need_cache(k_cache, v_cache, k_scale, v_scale)
    P, ps, Hkv, d = k_cache.shape
    _need(src, torch.int32, 1, "src")
    _need_ints(src.shape, "dst", dst)
    with _device_of(k_cache, v_cache, k_scale, v_scale, src, dst):
        _check(_lib.fa_cache_copy_pages(_ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
                                        eb, _ptr(src), _ptr(dst), src.shape[0], P, Hkv, d, ps,
                                        _stream(stream)), "fa_cache_copy_pages")


def cache_collect_workspace_bytes(num_pages) -> int:
    return int(_lib.fa_cache_collect_workspace_bytes(int(num_pages)))


def cache_collect(block_table, seq_lens, free_pages, free_count, page_size=16, workspace=None,
                  stream=None):
    """The pages that no sequence uses, descending, into free_pages [P] and free_count [1]
    (int32, device), from block_table [S,maxp] and seq_lens [S]."""
    if stream is not None:
        return _inside(cache_collect, stream, locals())
    _need(block_table, torch.int32, 2, "block_table")
    _need(free_pages, torch.int32, 1, "free_pages")
    S, maxp = block_table.shape
    P = free_pages.shape[0]
    _need_ints((S,), "seq_lens", seq_lens)
    _need_ints((1,), "free_count", free_count)
    workspace = _bytes_of(workspace, cache_collect_workspace_bytes(P), block_table)
    with _device_of(block_table, seq_lens, free_pages, free_count,
                    workspace):
        _check(_lib.fa_cache_collect(_ptr(block_table), _ptr(seq_lens), S, maxp, P,
                                     int(page_size), _ptr(free_pages), _ptr(free_count),
                                     _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     _stream(stream)), "fa_cache_collect")


def cache_compact_workspace_bytes(num_pages) -> int:
    return int(_lib.fa_cache_compact_workspace_bytes(int(num_pages)))


def cache_compact(k_cache, v_cache, block_table, seq_lens, block_table_out, free_pages, free_count,
                  k_scale=None, v_scale=None, workspace=None, stream=None):
    """Moves the pages in use to the cache's front.  caches [P,16,Hkv,d] (bf16, or E4M3 with
    scales), block_table [S,maxp], seq_lens [S] int32 -> writes block_table_out [S,maxp] (may
    be block_table), free_pages [P], free_count [1]."""
    if stream is not None:
        return _inside(cache_compact, stream, locals())
    k_cache, v_cache, eb = _need_cache(k_cache, v_cache, k_scale, v_scale)
    P, ps, Hkv, d = k_cache.shape
    _need(block_table, torch.int32, 2, "block_table")
    S, maxp = block_table.shape
    _need_ints((S,), "seq_lens", seq_lens)
    _need_ints((S, maxp), "block_table_out", block_table_out)
    _need_ints((P,), "free_pages", free_pages)
    _need_ints((1,), "free_count", free_count)
    workspace = _bytes_of(workspace, cache_compact_workspace_bytes(P), k_cache)
    with _device_of(k_cache, v_cache, k_scale, v_scale,
                    block_table, seq_lens, block_table_out,
                    free_pages, free_count, workspace):
        _check(_lib.fa_cache_compact(_ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
                                     eb, _ptr(block_table), _ptr(seq_lens), S,
                                     _ptr(block_table_out), _ptr(free_pages), _ptr(free_count), P,
                                     Hkv, d, ps, maxp, _ptr(workspace),
                                     workspace.numel() * workspace.element_size(),
                                     _stream(stream)), "fa_cache_compact")


def _on_device_of(stream):
    return _same_device if stream is None else torch.cuda.device(stream.device)


def selftest_watchdog(stream=None) -> int:
    """Launch the watchdog diagnostic (a wait that must time out); read the
    result with check_device_error()."""
    with _on_device_of(stream):
        return int(_lib.fa_selftest_watchdog(_stream(stream)))


def check_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error status of
    its device (of the current one without a stream)."""
    with _on_device_of(stream):
        return int(_lib.fa_check_device_error(_stream(stream)))
